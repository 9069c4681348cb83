"""The paged-cache operators: cases, their plain forms and what each has to move.

append  new tokens' keys and values into a paged cache, with the rotary positions applied on the way
decode  attention of one new token of each sequence over the paged cache
sparse  the same over the pages that a per-page score selects for each token and kv head
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One user, one token: the smallest append of a serving loop, nothing but latency.
        dict(name="append_one", op="append", seqs=1, shortest=700, longest=700, new=1, padding=0, q_heads=32, kv_heads=4,
             dim=128, rot=128, interleaved=False, page=16, dtype="bf16"),
        # A full decoding batch, padded to its graph's size.
        dict(name="append_batch", op="append", seqs=251, shortest=17, longest=8191, new=1, padding=5, q_heads=32,
             kv_heads=8, dim=128, rot=64, interleaved=True, page=64, dtype="bf16"),
        # Prompts of a few users written in one pass.
        dict(name="append_prompts", op="append", seqs=4, shortest=4099, longest=16384, new=16384, padding=0, q_heads=32,
             kv_heads=4, dim=128, rot=128, interleaved=False, page=64, dtype="bf16"),
        # A small float32 model; pieces of a prompt behind a cached prefix, short pages.
        dict(name="append_f32", op="append", seqs=3, shortest=700, longest=2047, new=301, padding=2, q_heads=8, kv_heads=2,
             dim=64, rot=32, interleaved=False, page=8, dtype="f32"),
        # One user's reply to a short question.
        dict(name="decode_one_short", op="decode", seqs=1, shortest=333, longest=333, q_heads=32, kv_heads=4, dim=128,
             page=16, dtype="bf16"),
        # One user with a long document.
        dict(name="decode_one_32k", op="decode", seqs=1, shortest=32768, longest=32768, q_heads=32, kv_heads=4, dim=128,
             page=16, dtype="bf16"),
        # A mixed decoding batch: most sequences short, a few long.
        dict(name="decode_batch", op="decode", seqs=64, shortest=1, longest=16384, q_heads=32, kv_heads=8, dim=128,
             page=32, dtype="bf16"),
        # Long documents of several users: the bandwidth case.
        dict(name="decode_long", op="decode", seqs=8, shortest=131071, longest=131071, q_heads=32, kv_heads=4, dim=128,
             page=64, dtype="bf16"),
        # A small float32 model.
        dict(name="decode_f32", op="decode", seqs=3, shortest=99, longest=4097, q_heads=8, kv_heads=2, dim=64, page=16,
             dtype="f32"),
        # One user with a very long context, a 64th of whose pages is read.
        dict(name="sparse_256k", op="sparse", seqs=1, shortest=262144, longest=262144, select=64, q_heads=32, kv_heads=8,
             dim=128, page=64, dtype="bf16"),
        # A mixed batch; the shorter sequences have no more pages than are selected.
        dict(name="sparse_batch", op="sparse", seqs=32, shortest=100, longest=65536, select=200, q_heads=32, kv_heads=4,
             dim=128, page=16, dtype="bf16"),
        # A small float32 model.
        dict(name="sparse_f32", op="sparse", seqs=2, shortest=900, longest=5001, select=20, q_heads=8, kv_heads=2, dim=64,
             page=16, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "sparse"])
    q_heads, kv_heads = rng.choice([(32, 4), (32, 8), (8, 2), (8, 8), (12, 4), (32, 2), (8, 1), (1, 1)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, 128, 96, 80])
    case = dict(op=op, seqs=_log_int(rng, 1, 256), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                page=rng.choice([8, 16, 32, 64, 128]), dtype=dtype)
    row = kv_heads * dim * (4 if dtype == "f32" else 2)
    if op == "append":
        most = 300_000_000 // (q_heads * dim * (4 if dtype == "f32" else 2))
        case["new"] = rng.choice([1, _log_int(rng, 2, 16384)])
        case["longest"] = _log_int(rng, 1, 16384)
        case["seqs"] = max(1, min(case["seqs"], most // min(case["new"], case["longest"]), 250_000_000 // (row * case["longest"])))
        case["padding"] = rng.choice([0, 0, rng.randint(1, 9)])
        case["rot"] = rng.choice([dim, dim, dim // 2, 16])
        case["interleaved"] = rng.choice([False, True])
    else:
        case["longest"] = _log_int(rng, 1, 131072)
        case["seqs"] = max(1, min(case["seqs"], 1_000_000_000 // (row * case["longest"])))
    if op == "sparse":
        case["select"] = _log_int(rng, 4, 256)
    case["shortest"] = rng.choice([case["longest"], _log_int(rng, 1, case["longest"])])
    return case


def _lengths(case):
    """The sequences' lengths: spread evenly over the logarithm of their range."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** (i / (n - 1)))))) for i in range(n)]


def _new(case):
    return [min(case["new"], n) for n in _lengths(case)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dtype, page, dim = DTYPES[case["dtype"]], case["page"], case["dim"]
    hq, hkv, n = case["q_heads"], case["kv_heads"], case["seqs"]
    lens = torch.tensor(_lengths(case))[torch.randperm(n, generator=host)]
    pages = (lens + page - 1) // page
    width, total = int(pages.max()), int(pages.sum())
    # Pages lie anywhere in the cache, as after hours of serving; some belong to nobody. A row of the table is padded with 0.
    n_pages = total + 7
    ids = torch.randperm(n_pages, generator=host)[:total].to(torch.int32)
    table = torch.zeros(n, width, dtype=torch.int32)
    table[torch.arange(width) < pages[:, None]] = ids

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    # Keys of one page resemble one another (neighbouring tokens): a page's own centre plus noise.
    k_cache, v_cache = randn(n_pages, hkv, page, dim).mul_(0.75), randn(n_pages, hkv, page, dim)
    k_cache.add_(randn(n_pages, hkv, 1, dim), alpha=0.65)
    s = dict(case=case, k_cache=k_cache, v_cache=v_cache, table=table.to(dev), lens=lens.to(torch.int32).to(dev))
    if case["op"] != "decode":
        s["bounds"] = torch.stack((k_cache.amin(2), k_cache.amax(2)), 2)  # [n_pages, kv heads, 2, dim]
    if case["op"] == "append":
        new = torch.minimum(lens, torch.tensor(case["new"]))
        seq = torch.repeat_interleave(torch.arange(n), new)
        start = torch.cumsum(new, 0) - new
        pos = torch.arange(seq.numel()) - start[seq] + (lens - new)[seq]
        pad = torch.full((case["padding"],), -1)
        s["token_seq"] = torch.cat((seq, pad)).to(torch.int32).to(dev)
        s["token_pos"] = torch.cat((pos, torch.zeros_like(pad))).to(torch.int32).to(dev)
        # One projection's output holds a token's queries, keys and values side by side.
        s["qkv"] = randn(s["token_seq"].numel(), hq + 2 * hkv, dim)
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        angle = torch.arange(int(lens.max()), dtype=torch.float64)[:, None] * freq
        s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float().to(dev)
    else:
        s["q"] = randn(n, hq, dim)
    if own:
        from split_kv_lse_splitkv_b200 import PagedKV
        s["handle"] = PagedKV(hq, hkv, dim, page, max_seqs=n, max_pages=width, k_cache=k_cache, v_cache=v_cache,
                              k_bounds=s.get("bounds"))
    return s


def _split(s):
    hq, hkv = s["case"]["q_heads"], s["case"]["kv_heads"]
    return s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]


def run(s):
    case = s["case"]
    if own:
        kv = s["handle"]
        if case["op"] == "append":
            q, k, v = _split(s)
            q = kv.append(k, v, s["table"], s["token_seq"], s["token_pos"], q=q, rope=s["rope"],
                          interleaved=case["interleaved"])
            return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], bounds=s["bounds"])
        if case["op"] == "decode":
            o, lse = kv.decode(s["q"], s["table"], s["lens"])
            return dict(o=o, lse=lse)
        pages = kv.select(s["q"], s["table"], s["lens"], case["select"], keep_first=1, keep_last=1)
        o, lse = kv.decode(s["q"], s["table"], s["lens"], pages=pages)
        return dict(o=o, lse=lse, pages=pages)
    if case["op"] == "append":
        return _append(s)
    return _decode(s) if case["op"] == "decode" else _sparse(s)


# ------------------------------------------------------------------ the plain forms

def _rotate(x, cos, sin, interleaved):
    """x [N, H, d] in 32 bits, cos and sin [N, 1, R/2]."""
    r = 2 * cos.shape[-1]
    turned, rest = x[..., :r], x[..., r:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :r // 2], turned[..., r // 2:])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((y, rest), -1)


def _append(s):
    case, page = s["case"], s["case"]["page"]
    dtype = DTYPES[case["dtype"]]
    q, k, v = _split(s)
    seq, pos = s["token_seq"].long(), s["token_pos"].long()
    real = seq >= 0
    cs = s["rope"][pos].unsqueeze(1)
    cos, sin = cs.chunk(2, -1)
    turned = _rotate(torch.cat((q, k), 1).float(), cos, sin, case["interleaved"]).to(dtype)
    turned = torch.where(real[:, None, None], turned, torch.cat((q, k), 1))  # a padding row's queries stay as they are
    hq = case["q_heads"]
    seq, pos = seq[real], pos[real]
    at = s["table"][seq, pos // page].long()
    s["k_cache"][at, :, pos % page] = turned[real, hq:]
    s["v_cache"][at, :, pos % page] = v[real]
    # A page that was written: the bounds of its keys up to the last new one.
    last = torch.full((s["k_cache"].shape[0],), -1, dtype=torch.int64, device=at.device).scatter_reduce(0, at, pos % page, "amax")
    written = (last >= 0).nonzero()[:, 0]
    held = (torch.arange(page, device=at.device) <= last[written][:, None])[:, None, :, None]
    keys = s["k_cache"][written].float()
    low = torch.where(held, keys, math.inf).amin(2)
    high = torch.where(held, keys, -math.inf).amax(2)
    s["bounds"][written] = torch.stack((low, high), 2).to(dtype)
    return dict(q=turned[:, :hq], k_cache=s["k_cache"], v_cache=s["v_cache"], bounds=s["bounds"])


def _attend(q, k, v, seen):
    """q [B, Hq, d], k and v [B, Hkv, n, d] of any type, seen [B, 1 or Hkv, n]; in 32 bits."""
    b, hq, d = q.shape
    hkv = k.shape[1]
    qg = q.float().view(b, hkv, hq // hkv, d)
    score = torch.matmul(qg, k.float().transpose(2, 3)) * (1.0 / math.sqrt(d))
    score = torch.where(seen[:, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight, torch.where(seen[..., None], v, 0).float()) / total
    lse = top + torch.log(total)
    return o.view(b, hq, d).to(q.dtype), lse.view(b, hq)


def _decode(s):
    n, hkv, d = s["q"].shape[0], s["case"]["kv_heads"], s["case"]["dim"]
    at = s["table"].long()
    k = s["k_cache"][at].transpose(1, 2).reshape(n, hkv, -1, d)
    v = s["v_cache"][at].transpose(1, 2).reshape(n, hkv, -1, d)
    seen = torch.arange(k.shape[2], device=k.device) < s["lens"][:, None]
    o, lse = _attend(s["q"], k, v, seen[:, None])
    return dict(o=o, lse=lse)


def _sparse(s):
    case, page, d, hkv = s["case"], s["case"]["page"], s["case"]["dim"], s["case"]["kv_heads"]
    n, width = s["table"].shape
    # Scores in 64 bits: a rounding may not decide which page comes in.
    q = s["q"].double().view(n, hkv, -1, d)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    bounds = s["bounds"][s["table"].long()].double()  # [B, width, kv heads, 2, d]
    score = (bounds[..., 1, :] * up[:, None]).sum(-1) + (bounds[..., 0, :] * down[:, None]).sum(-1)
    count = (s["lens"].long() + page - 1) // page
    index = torch.arange(width, device=score.device)[None, :, None]
    score = torch.where((index < 1) | (index >= count[:, None, None] - 1), math.inf, score)
    score = torch.where(index < count[:, None, None], score, -math.inf)
    order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["select"]].transpose(1, 2)
    taken = torch.where(order < count[:, None, None], order, width).sort(-1).values  # [B, kv heads, select], ascending
    real = taken < width
    taken = torch.where(real, taken, 0)
    at = torch.gather(s["table"].long()[:, None].expand(n, hkv, width), 2, taken)
    head = torch.arange(hkv, device=at.device)[None, :, None]
    k = s["k_cache"][at, head].reshape(n, hkv, -1, d)
    v = s["v_cache"][at, head].reshape(n, hkv, -1, d)
    key = taken[..., None] * page + torch.arange(page, device=at.device)
    seen = (real[..., None] & (key < s["lens"][:, None, None, None])).flatten(2)
    o, lse = _attend(s["q"], k, v, seen)
    pages = torch.where(real, taken, -1).to(torch.int32)
    if pages.shape[2] < case["select"]:
        pages = torch.cat((pages, pages.new_full((n, hkv, case["select"] - pages.shape[2]), -1)), 2)
    return dict(o=o, lse=lse, pages=pages)


# ------------------------------------------------------------------ what each has to move, and its values in 64 bits

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    hq, hkv, d, page, n = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["seqs"]
    lens = _lengths(case)
    if case["op"] == "append":
        new = _new(case)
        rows = sum(new)
        touched = sum((l - 1) // page - (l - m) // page + 1 for l, m in zip(lens, new))
        before = sum((l - m) % page for l, m in zip(lens, new))  # keys that a page's bounds take in and that were there
        nbytes = (rows * (2 * hq + 4 * hkv) + case["padding"] * 2 * hq + touched * 2 * hkv + before * hkv) * d * e
        nbytes += min(rows, max(lens)) * case["rot"] * 4 + (rows + case["padding"]) * 8 + touched * 4
        return dict(bytes=nbytes, flops=rows * (hq + hkv) * case["rot"] * 3)
    small = 2 * n * hq * d * e + 4 * n * hq + 4 * n
    if case["op"] == "decode":
        return dict(bytes=2 * sum(lens) * hkv * d * e + small + 4 * sum(-(-l // page) for l in lens),
                    flops=4 * sum(lens) * hq * d)
    counts = [-(-l // page) for l in lens]
    taken = [min(c, case["select"]) for c in counts]
    keys = sum(t * page - (c * page - l) for t, c, l in zip(taken, counts, lens))  # the last page is always in
    nbytes = 2 * keys * hkv * d * e + 2 * sum(counts) * hkv * d * e + small + 4 * sum(counts) + 4 * n * hkv * case["select"]
    return dict(bytes=nbytes, flops=4 * keys * hq * d + 4 * sum(counts) * hkv * d + n * hq * d)


def exact(case, seed):
    s = prepare(case, seed)
    page, d, hq, hkv = case["page"], case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "append":
        q, k, v = (x.double() for x in _split(s))
        half = case["rot"] // 2
        lo = torch.arange(half, device=q.device) * (2 if case["interleaved"] else 1)
        hi = lo + (1 if case["interleaved"] else half)
        real = s["token_seq"] >= 0
        z = torch.complex(s["rope"][s["token_pos"].long(), :half].double(), s["rope"][s["token_pos"].long(), half:].double())
        z = torch.where(real[:, None], z, torch.ones_like(z))[:, None]
        for x in (q, k):
            turned = torch.complex(x[..., lo], x[..., hi]) * z
            x[..., lo], x[..., hi] = turned.real, turned.imag
        kc, vc, bounds = s["k_cache"].double(), s["v_cache"].double(), s["bounds"].double()
        slot = s["table"][s["token_seq"].long().clamp(min=0), s["token_pos"].long() // page].long() * page + s["token_pos"].long() % page
        rows_k, rows_v = kc.transpose(1, 2).reshape(-1, hkv, d), vc.transpose(1, 2).reshape(-1, hkv, d)
        rows_k[slot[real]], rows_v[slot[real]] = k[real], v[real]
        kc, vc = (x.view(-1, page, hkv, d).transpose(1, 2).contiguous() for x in (rows_k, rows_v))
        # By the number of keys that a written page holds now: each count's pages at once.
        held = torch.zeros(kc.shape[0], dtype=torch.int64, device=kc.device)
        held.scatter_reduce_(0, slot[real] // page, slot[real] % page + 1, "amax")
        for m in range(1, page + 1):
            at = (held == m).nonzero()[:, 0]
            if at.numel():
                part = kc[at, :, :m]
                bounds[at, :, 0], bounds[at, :, 1] = part.amin(2), part.amax(2)
        return dict(q=q, k_cache=kc, v_cache=vc, bounds=bounds)
    o = torch.zeros(case["seqs"], hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(case["seqs"], hq, dtype=torch.float64, device=s["q"].device)
    for b in range(case["seqs"]):
        length = int(s["lens"][b])
        count = -(-length // page)
        at = s["table"][b, :count].long()
        for g in range(hkv):
            q = s["q"][b, g * (hq // hkv):(g + 1) * (hq // hkv)].double()
            chosen = torch.arange(count, device=at.device)
            if case["op"] == "sparse" and count > case["select"]:
                box = s["bounds"][at, g].double()
                reach = torch.maximum(q[:, None] * box[None, :, 0], q[:, None] * box[None, :, 1]).sum((0, 2))
                reach[0] = reach[count - 1] = math.inf
                chosen = torch.argsort(reach, descending=True, stable=True)[:case["select"]].sort().values
            keys = (chosen[:, None] * page + torch.arange(page, device=at.device)).flatten()
            inside = keys < length
            k = s["k_cache"][at[chosen], g].double().flatten(0, 1)[inside]
            v = s["v_cache"][at[chosen], g].double().flatten(0, 1)[inside]
            score = q @ k.T / math.sqrt(d)
            lse[b, g * (hq // hkv):(g + 1) * (hq // hkv)] = torch.logsumexp(score, 1)
            o[b, g * (hq // hkv):(g + 1) * (hq // hkv)] = torch.softmax(score, 1) @ v
    return dict(o=o, lse=lse, pages=None) if case["op"] == "sparse" else dict(o=o, lse=lse)
