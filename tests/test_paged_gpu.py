"""The paged-cache operators on the GPU against the float64 oracle.

Tolerances (derived, per element). A float32 dot product of d terms, in any order, is off by at most
d 2^-23 sum|q_i k_i| (bf16 products are exact in float32; float32 products are formed from three products of
11-bit halves, what is left out is below 2^-20 of each product). With R = the largest scale * sum|q_i k_i| of a row
(the oracle's `reach`), a score is off by e = (d 2^-23 + 2^-20) R, and by another 2^-22 of itself (scaling, the
reference point, the exponential's argument). Its weight is then off by e' = e + 2^-21 R + 2^-20 relative (2^-22 for
the exponential, 2^-16 for the weights that enter the value product, which are split into two bf16 halves), the
sums of n terms by n 2^-23 more. So
    |o - ref| <= step |ref| + (2 e' + 2^-16 + 2 n 2^-23) sum_j p_j |v_j|       (step: eps/2 of the output type)
    |lse - ref| <= e' + n 2^-23 + 2^-23 |ref|.
Rotations: two products and a sum in float32 (3 roundings of 2^-24 on |x| + |y|), then one rounding to the type.
"""
import gc
import threading

import numpy as np
import pytest
import torch

from oracle import paged as OP

pytestmark = pytest.mark.gpu
B = pytest.importorskip("split_kv_lse_splitkv_b200.binding", reason="libsplitkv.so not built")
from split_kv_lse_splitkv_b200.paged import PagedKV, rope_table  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Case:
    """A cache with sequences of the given lengths at random pages. Whatever no sequence may read is NaN or a page
    number out of range."""

    def __init__(self, lens, hq, hkv, d, page, dtype=BF, seed=0, order="heads", spare=3, amp=1.0, width=None, q_gap=0):
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hkv, self.d, self.page, self.dtype = hq, hkv, d, page, dtype
        self.lens_l = [int(x) for x in lens]
        counts = [-(-n // page) for n in self.lens_l]
        total = sum(counts) + spare
        width = max(1, max(counts)) if width is None else width
        ids = torch.randperm(total, generator=g)
        table = torch.full((len(lens), width), -5, dtype=torch.int32)  # entries past the length: not to be read
        table[:, -1] = 1 << 30
        k = torch.full((total, hkv, page, d), float("nan"))
        v = torch.full((total, hkv, page, d), float("nan"))
        at = 0
        for b, n in enumerate(self.lens_l):
            for e in range(counts[b]):
                p = int(ids[at])
                at += 1
                table[b, e] = p
                m = min(page, n - e * page)
                k[p, :, :m] = torch.randn(hkv, m, d, generator=g)
                v[p, :, :m] = torch.randn(hkv, m, d, generator=g)
        self.table = table.cuda()
        self.lens = torch.tensor(self.lens_l, dtype=torch.int32).cuda()
        self.k, self.v = self._lay(k.to(dtype), order), self._lay(v.to(dtype), order)
        wide = torch.randn(len(lens), hq + q_gap, d, generator=g).mul(amp).to(dtype).cuda()
        self.q = wide[:, :hq]
        self.kv = PagedKV(hq, hkv, d, page, max_seqs=max(1, len(lens)), max_pages=width, k_cache=self.k, v_cache=self.v)

    @staticmethod
    def _lay(x, order):
        x = x.cuda()
        if order == "heads":  # [pages, heads, positions, d]
            return x.contiguous()
        if order == "positions":  # a view of [pages, positions, heads, d]
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if order == "outer":  # a view of [heads, pages, positions, d]
            return x.transpose(0, 1).contiguous().transpose(0, 1)
        wide = torch.full((x.shape[0], x.shape[1] + 1, x.shape[2] + 1, x.shape[3] + 16), float("nan"), dtype=x.dtype,
                          device=x.device)
        wide[:, :-1, :-1, :-16] = x
        return wide[:, :-1, :-1, :-16]  # "gaps": rows, positions and heads apart

    def oracle(self, pages=None, q=None, lens=None):
        return OP.decode(f64(self.q if q is None else q), f64(self.k), f64(self.v), self.table.cpu().numpy(),
                         self.lens_l if lens is None else lens, 1 / np.sqrt(self.d), pages)

    def check(self, o, lse, ref, n=None):
        ro, rl, spread, reach = ref
        assert o.dtype == self.dtype and lse.dtype == F32
        n = max(self.lens_l) if n is None else n
        e = (self.d * 2.0**-23 + 2.0**-20) * reach + 2.0**-21 * reach + 2.0**-20
        o, lse = f64(o), f64(lse)
        empty = np.isneginf(rl)
        assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
        lim = half_step(self.dtype) * np.abs(ro) + (2 * e[..., None] + 2.0**-16 + 2 * n * 2.0**-23) * spread + 1e-30
        err = np.abs(o - ro)
        worst = float((err / lim).max()) if err.size else 0.0
        assert np.isfinite(o).all() and worst <= 1, f"o: {worst:.3g} of its bound"
        full = ~empty
        lerr = np.abs(lse[full] - rl[full])
        llim = (e + n * 2.0**-23)[full] + 2.0**-23 * np.abs(rl[full])
        assert (lerr <= llim).all(), f"lse: {float((lerr / llim).max()):.3g} of its bound"
        print(f"[parity] o {worst:.3g}, lse {float((lerr / llim).max()) if lerr.size else 0:.3g} of the bound")


EDGE_LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 300, 0, 1000]


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d", [(32, 4, 128), (8, 8, 64), (12, 4, 96), (16, 1, 80), (40, 1, 128), (1, 1, 8), (6, 2, 24),
                                      (34, 2, 112)])
@pytest.mark.parametrize("page", [1, 8, 16, 64])
def test_decode(dtype, hq, hkv, d, page):
    c = Case(EDGE_LENS, hq, hkv, d, page, dtype, seed=page + d)
    o, lse = c.kv.decode(c.q, c.table, c.lens)
    c.kv.check_status()
    c.check(o, lse, c.oracle())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", ["positions", "outer", "gaps"])
def test_decode_cache_orders(dtype, order):
    c = Case([5, 700, 0, 64], 8, 2, 64, 32, dtype, order=order, q_gap=3)
    o, lse = c.kv.decode(c.q, c.table, c.lens)
    c.kv.check_status()
    c.check(o, lse, c.oracle())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,hq,hkv,d,page", [([20011], 4, 2, 128, 16), ([1], 32, 4, 128, 16), ([9001, 3, 5000], 8, 1, 64, 128),
                                                ([37] * 200, 8, 4, 64, 16), ([777] * 3 + [0] * 5, 2, 2, 128, 1024),
                                                ([0], 4, 4, 64, 16), ([0] * 7, 4, 1, 64, 16)])
def test_decode_lengths(dtype, lens, hq, hkv, d, page):
    c = Case(lens, hq, hkv, d, page, dtype, seed=3)
    o, lse = c.kv.decode(c.q, c.table, c.lens)
    c.kv.check_status()
    c.check(o, lse, c.oracle())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_large_scores(dtype):
    # Queries of 30 times the size: one key carries a row, the running maximum moves often.
    c = Case([2, 40, 1500], 16, 2, 128, 16, dtype, amp=30.0)
    o, lse = c.kv.decode(c.q, c.table, c.lens)
    c.check(o, lse, c.oracle())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_rising_and_infinite_scores(dtype):
    # Keys that grow along the sequence (every part has a larger maximum), and keys whose score is -inf.
    c = Case([3000, 50], 4, 1, 64, 16, dtype)
    flat = c.table[0].long()
    for e in range(3000 // 16):
        c.k[flat[e]] *= 1 + e / 40
    c.q[1].fill_(1.0)
    rows = c.table[1].long()
    c.k[rows[0], :, :3] = -float("inf")
    ref = c.oracle()
    o, lse = c.kv.decode(c.q, c.table, c.lens)
    ro, rl, spread, reach = ref
    reach[~np.isfinite(reach)] = 8 * 8  # the -inf keys take no part
    c.check(o, lse, (ro, rl, spread, reach))
    # Only -inf scores: an empty row.
    short = torch.tensor([0, 3], dtype=torch.int32).cuda()
    o, lse = c.kv.decode(c.q, c.table, short)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_decode_is_deterministic_and_leaves_its_scratch_ready():
    c = Case([5000, 31, 0, 2222], 32, 4, 128, 16)
    first = [x.clone() for x in c.kv.decode(c.q, c.table, c.lens)]
    for _ in range(5):
        again = c.kv.decode(c.q, c.table, c.lens)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    small = c.kv.decode(c.q[:1], c.table[:1], c.lens[:1])  # fewer sequences with the same object
    assert torch.allclose(small[1], first[1][:1], atol=1e-5)


def test_decode_several_tokens_of_a_sequence_share_its_row():
    c = Case([500], 8, 2, 64, 16, q_gap=0)
    n = 5
    table = c.table.expand(n, -1).contiguous()
    kv = PagedKV(8, 2, 64, 16, max_seqs=n, max_pages=table.shape[1], k_cache=c.k, v_cache=c.v)
    lens = torch.tensor([496, 497, 498, 499, 500], dtype=torch.int32).cuda()
    q = torch.randn(n, 8, 64, device="cuda").to(BF)
    o, lse = kv.decode(q, table, lens)
    ref = OP.decode(f64(q), f64(c.k), f64(c.v), table.cpu().numpy(), lens.tolist(), 1 / 8.0)
    c.check(o, lse, ref)


def test_decode_given_outputs_and_table_wider_than_used():
    c = Case([100, 30], 8, 2, 64, 16, width=50)
    o = torch.full((2, 8, 64), 7.0, device="cuda", dtype=BF)
    lse = torch.full((2, 8), 7.0, device="cuda")
    got = c.kv.decode(c.q, c.table, c.lens, o=o, lse=lse)
    assert got[0] is o and got[1] is lse
    c.check(o, lse, c.oracle())
    # A slice of a wider table.
    o2, lse2 = c.kv.decode(c.q, c.table[:, :7], c.lens)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_decode_offsets_past_32_bits():
    # Pages more than 2^32 elements into a cache of one 9 GB tensor each.
    page, hkv, d, n_pages = 64, 8, 128, (1 << 32) // (64 * 8 * 128) + 9
    k = torch.empty(n_pages, hkv, page, d, dtype=BF, device="cuda")
    v = torch.empty(n_pages, hkv, page, d, dtype=BF, device="cuda")
    table = torch.tensor([[n_pages - 1, 0, n_pages - 3]], dtype=torch.int32, device="cuda")
    for p in table[0].tolist():
        k[p].normal_()
        v[p].normal_()
    kv = PagedKV(16, hkv, d, page, max_seqs=1, max_pages=3, k_cache=k, v_cache=v)
    q = torch.randn(1, 16, d, device="cuda").to(BF)
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    o, lse = kv.decode(q, table, lens)
    at = table[0].long()
    ref = OP.decode(f64(q), f64(k[at]), f64(v[at]), np.array([[0, 1, 2]]), [150], 1 / np.sqrt(d))
    Case.check(type("C", (), dict(dtype=BF, d=d, lens_l=[150])), o, lse, ref)
    # Append and bounds at the far end too.
    kb = torch.zeros(n_pages, hkv, 2, d, dtype=BF, device="cuda")
    kv = PagedKV(16, hkv, d, page, max_seqs=1, max_pages=3, k_cache=k, v_cache=v, k_bounds=kb)
    new = torch.randn(1, hkv, d, device="cuda").to(BF)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.append(new, new, table, one, one + 150)
    assert torch.equal(k[n_pages - 3, :, 22], new[0]) and torch.equal(v[n_pages - 3, :, 22], new[0])
    assert torch.equal(kb[n_pages - 3, :, 1], k[n_pages - 3, :, :23].amax(1))
    kv.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (16, 4, 112), (4, 4, 40)])
def test_decode_wide_tables(dtype, hq, hkv, d):
    # A table for sequences of up to 32768 keys: the launch is made for much to read, whatever the lengths are.
    c = Case(EDGE_LENS + [5000], hq, hkv, d, 16, dtype, width=2048)
    o, lse = c.kv.decode(c.q, c.table, c.lens)
    ref = c.oracle()
    c.check(o, lse, ref)
    # So for lists: every page of every sequence, in lists of 2048.
    lists = np.full((len(c.lens_l), hkv, 2048), -1, dtype=np.int32)
    for b, n in enumerate(c.lens_l):
        lists[b, :, :-(-n // 16)] = np.arange(-(-n // 16))
    o, lse = c.kv.decode(c.q, c.table, c.lens, pages=torch.tensor(lists).cuda())
    c.check(o, lse, ref)
    c.kv.check_status()


# ------------------------------------------------------------------ decode over listed pages
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_in_several_launches(dtype):
    # Rows of 2^31 positions at 8 kv heads: two sequences a launch.
    c = Case([3000, 0, 17, 5000, 1], 16, 8, 64, 1024, dtype, width=(1 << 21) - 3, q_gap=1)
    c.check(*c.kv.decode(c.q, c.table, c.lens), c.oracle())
    pages = torch.full((5, 8, 2), -1, dtype=torch.int32)
    pages[0] = torch.tensor([0, 2])
    pages[2, :, 0], pages[4, :, 0] = 0, 0
    pages[3] = torch.tensor([1, 4])
    pages[3, 5] = torch.tensor([3, -1])
    c.check(*c.kv.decode(c.q, c.table, c.lens, pages=pages.cuda()), c.oracle(pages=pages.numpy()))
    c.kv.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [4, 16, 32])
def test_decode_listed_pages(dtype, page):
    c = Case([0, 1, 5 * page, 7 * page + 3, 40 * page - 1], 8, 2, 64, page, dtype)
    rng = np.random.default_rng(5)
    n_select = 9
    lists = np.full((5, 2, n_select), -1, dtype=np.int32)
    for b, n in enumerate(c.lens_l):
        for g in range(2):
            count = -(-n // page)
            take = rng.integers(0, min(count, n_select) + 1) if b != 2 else min(count, n_select)
            lists[b, g, :take] = np.sort(rng.permutation(count)[:take])
    o, lse = c.kv.decode(c.q, c.table, c.lens, pages=torch.tensor(lists).cuda())
    c.kv.check_status()
    c.check(o, lse, c.oracle(pages=lists))


@pytest.mark.parametrize("row", [[1, 1, -1], [2, 1, -1], [0, -1, 1], [4, -1, -1], [-2, -1, -1], [-1, -1, 0], [-1, 1 << 30, -1]])
def test_bad_page_lists_raise_the_status(row):
    c = Case([64], 2, 1, 64, 16)
    c.kv.decode(c.q, c.table, c.lens, pages=torch.tensor([[row]], dtype=torch.int32).cuda())
    assert c.kv.status_value() == B.DEV_BAD_PAGE
    c.kv.status.zero_()
    o, lse = c.kv.decode(c.q, c.table, c.lens)  # the scratch is as it was
    c.check(o, lse, c.oracle())


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_pages_and_lengths_raise_the_status(bad):
    c = Case([5000, 100], 8, 2, 64, 16)
    good = c.table.clone()
    c.table[0, 77] = bad
    c.kv.decode(c.q, c.table, c.lens)
    assert c.kv.status_value() == B.DEV_BAD_PAGE
    c.kv.decode(c.q, good, c.lens)  # sticky: the call does nothing, and says so
    assert c.kv.status_value() == B.DEV_BAD_PAGE
    c.kv.status.zero_()
    c.kv.decode(c.q, good, torch.tensor([5000, bad], dtype=torch.int32).cuda())
    assert c.kv.status_value() == B.DEV_BAD_LENGTH
    c.kv.status.zero_()
    o, lse = c.kv.decode(c.q, good, c.lens)
    c.table.copy_(good)
    c.check(o, lse, c.oracle())
    c.kv.check_status()


# ------------------------------------------------------------------ append
def run_append(lens, new, hq, hkv, d, page, dtype, rot, interleaved, order="heads", padding=(), with_q=True, bounds=True,
               seed=0):
    """Sequences of lens - new cached positions get `new` more each; padding: token indices given to nobody."""
    g = torch.Generator().manual_seed(seed)
    c = Case(lens, hq, hkv, d, page, dtype, seed=seed, order=order)
    kb = torch.full((c.k.shape[0], hkv, 2, d), 9.0, dtype=dtype, device="cuda") if bounds else None
    kv = PagedKV(hq, hkv, d, page, max_seqs=len(lens), max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    seq = [b for b, m in enumerate(new) for _ in range(m)]
    pos = [lens[b] - new[b] + i for b in range(len(lens)) for i in range(new[b])]
    for at in padding:
        seq.insert(at, -1)
        pos.insert(at, 1 << 30)
    n = len(seq)
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    rope = rope_table(max(lens) + 1, rot, device="cuda") if rot else None
    ok, ov = f64(c.k).copy(), f64(c.v).copy()
    obounds = None if kb is None else f64(kb).copy()
    # NaN lies where no key is: the rows of the new tokens themselves among them.
    qo = kv.append(k, v, c.table, torch.tensor(seq, dtype=torch.int32).cuda(), torch.tensor(pos, dtype=torch.int32).cuda(),
                   q=q if with_q else None, rope=rope, interleaved=interleaved)
    kv.check_status()
    ref_q = OP.append(f64(k), f64(v), c.table.cpu().numpy(), seq, pos, ok, ov, obounds, f64(q) if with_q else None,
                      None if rope is None else f64(rope), interleaved)
    step = half_step(dtype)

    def close(got, ref, size, name):
        got = f64(got)
        lim = step * np.abs(ref) + 3 * 2.0**-24 * size * (1 + step) + 1e-30
        assert (np.isnan(got) == np.isnan(ref)).all(), name
        ok_ = np.isnan(ref) | (np.abs(got - ref) <= lim)
        assert ok_.all(), f"{name}: {np.nanmax(np.abs(got - ref) / lim):.3g} of its bound"

    size = 2 * float(qkv.abs().max()) if rot else 0.0
    close(c.k, ok, size, "k_cache")
    assert np.array_equal(f64(c.v), ov, equal_nan=True)
    if with_q:
        close(qo, ref_q, size, "q")
    else:
        assert qo is None
    if kb is not None:
        # The bounds are exactly those of the keys that the cache holds.
        keys, touched = f64(c.k), {}
        for b, p in zip(seq, pos):
            if b >= 0:
                at = int(c.table[b, p // page])
                touched[at] = max(touched.get(at, 0), p % page)
        want = np.full(tuple(kb.shape), 9.0)
        for at, off in touched.items():
            want[at, :, 0], want[at, :, 1] = keys[at, :, :off + 1].min(1), keys[at, :, :off + 1].max(1)
        assert np.array_equal(f64(kb), want)
    return c


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d,rot", [(32, 4, 128, 128), (8, 2, 64, 32), (6, 2, 80, 80), (3, 1, 24, 6), (8, 8, 96, 10), (1, 1, 8, 8),
                                          (4, 2, 64, 2), (4, 2, 64, 0), (5, 5, 112, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, hq, hkv, d, rot, interleaved):
    run_append([1, 5, 40, 33, 16, 100], [1, 5, 1, 2, 16, 70], hq, hkv, d, 16, dtype, rot, interleaved, seed=d + rot)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 2, 8, 64, 1024])
@pytest.mark.parametrize("order", ["heads", "positions", "gaps"])
def test_append_pages_and_orders(dtype, page, order):
    run_append([3, 130, 64, 7, 9], [3, 100, 1, 0, 9], 8, 2, 64, page, dtype, 64, False, order=order)


def test_append_padding_and_options():
    run_append([20, 9], [5, 3], 8, 2, 64, 8, BF, 64, False, padding=(0, 1, 4, 6, 12))
    run_append([20, 9], [5, 3], 8, 2, 64, 8, BF, 64, True, with_q=False)
    run_append([20, 9], [5, 3], 8, 2, 64, 8, BF, 0, False, bounds=False)
    run_append([20, 9], [0, 0], 8, 2, 64, 8, BF, 64, False, padding=(0, 1, 2))  # padding only
    run_append([50], [50], 8, 2, 64, 8, BF, 64, False, padding=tuple(range(0, 90, 2)))  # padding between any two
    run_append([2100, 300], [2000, 290], 8, 2, 64, 32, BF, 64, False)
    run_append([7] * 300, [1] * 300, 8, 2, 64, 16, F32, 64, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d,rot,interleaved", [(32, 4, 128, 128, False), (3, 1, 128, 64, True), (40, 10, 64, 64, False),
                                                      (1, 1, 16, 16, False), (6, 2, 80, 0, False), (8, 8, 112, 112, True)])
@pytest.mark.parametrize("page", [4, 64])
def test_append_many_tokens(dtype, hq, hkv, d, rot, interleaved, page):
    # Enough rows that they stream one by one, with their bounds in a second launch: sequences that begin and end inside
    # pages, padding inside and behind them.
    n = 148 * 32 * (32 // max(1, (d * (2 if dtype == BF else 4) + 31) // 32)) // (hq + 2 * hkv) + 100
    lens, new = [n // 2 + 3, 5, n // 2, 70], [n // 2 - 9, 5, n // 2, 1]
    run_append(lens, new, hq, hkv, d, page, dtype, rot, interleaved, padding=(0, 7, 40, 41, 300), seed=d)


@pytest.mark.parametrize("rot", [64, 10])
@pytest.mark.parametrize("width", [600, 3000])
def test_append_padded_batch(width, rot):
    # Rows of `width` tokens, the shorter ones filled up: the token before a run of padding is looked for behind it.
    new = [width, 1, 255, 256, 257, width - 1]
    padding, at = [], 0
    for n in new:
        padding += range(at + n, at + width)
        at += width
    run_append([n + 5 for n in new], new, 8, 2, 64, 16, BF, rot, False, padding=padding)
    # A page's tokens on both sides of a run.
    run_append([width + 20], [width + 20], 8, 2, 64, 16, BF, rot, False, padding=range(5, 5 + 2 * width))


@pytest.mark.parametrize("rot", [64, 10])
@pytest.mark.parametrize("tokens", [2, 9000])
@pytest.mark.parametrize("run", [31, 256, 5000])
def test_append_order_is_checked_across_padding(run, tokens, rot):
    c = Case([tokens], 8, 2, 64, 16)
    kv = PagedKV(8, 2, 64, 16, max_seqs=1, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v)
    pos = torch.arange(tokens, dtype=torch.int32)
    pos = torch.cat((pos[:tokens // 2], torch.zeros(run, dtype=torch.int32), pos[tokens // 2 :]))
    seq = torch.zeros(tokens + run, dtype=torch.int32)
    seq[tokens // 2 : tokens // 2 + run] = -1
    x = torch.zeros(tokens + run, 2, 64, dtype=BF, device="cuda")
    rope = rope_table(tokens, rot)
    kv.append(x, x, c.table, seq.cuda(), pos.cuda(), rope=rope)
    assert kv.status_value() == 0
    pos[tokens // 2 + run] = tokens // 2 - 1
    kv.append(x, x, c.table, seq.cuda(), pos.cuda(), rope=rope)
    assert kv.status_value() == B.DEV_TOKEN_ORDER


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d,rot", [(32, 4, 80, 40), (8, 2, 128, 24), (6, 2, 64, 8), (4, 1, 128, 4), (3, 3, 24, 12),
                                          (8, 8, 112, 104), (1, 1, 8, 4)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page", [4, 64])
def test_append_narrow_rotations(dtype, hq, hkv, d, rot, interleaved, page):
    # Half of the rotated channels is not a multiple of 16 bytes: pieces of 8, or channel by channel. Few tokens and many.
    run_append([1, 5, 40, 33, 16, 100], [1, 5, 1, 2, 16, 70], hq, hkv, d, page, dtype, rot, interleaved, padding=(3, 4),
               seed=d + rot)
    rows = max(1, 32 // max(1, d * (2 if dtype == BF else 4) // 16))
    n = 148 * 32 * rows // (hq + 2 * hkv) + 100
    run_append([n // 2 + 3, 5, n // 2], [n // 2 - 9, 5, n // 2], hq, hkv, d, page, dtype, rot, interleaved,
               padding=(0, 7, 40, 300), seed=rot)


def test_append_many_tokens_orders_and_options():
    run_append([3000, 2000], [2500, 2000], 8, 2, 128, 32, BF, 128, False, order="positions")
    run_append([3000, 2000], [2500, 2000], 8, 2, 128, 32, F32, 128, True, order="gaps")
    run_append([9000], [9000], 8, 2, 128, 1024, BF, 128, False, with_q=False)
    run_append([9000], [8990], 8, 2, 128, 1, BF, 128, False, with_q=False)
    run_append([9000], [8990], 8, 2, 128, 16, BF, 64, False, bounds=False)


@pytest.mark.parametrize("what,bit", [("order", B.DEV_TOKEN_ORDER), ("seq", B.DEV_BAD_TOKEN), ("pos", B.DEV_BAD_TOKEN),
                                      ("page", B.DEV_BAD_PAGE)])
def test_append_many_tokens_bad_ones_raise_the_status(what, bit):
    n = 9000
    c = Case([n], 8, 2, 128, 16)
    kb = torch.zeros(c.k.shape[0], 2, 2, 128, dtype=BF, device="cuda")
    kv = PagedKV(8, 2, 128, 16, max_seqs=1, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table = c.table.clone()
    if what == "order":
        pos[5000] = 4999
    elif what == "seq":
        seq[5000:] = 1
    elif what == "pos":
        pos[n - 1] = table.shape[1] * 16
    else:
        table[0, 300] = c.k.shape[0]
    x = torch.zeros(n, 2, 128, dtype=BF, device="cuda")
    kv.append(x, x, table, seq, pos, q=torch.zeros(n, 8, 128, dtype=BF, device="cuda"), rope=rope_table(n + 100, 128))
    assert kv.status_value() == bit


@pytest.mark.parametrize("what,bit", [("order", B.DEV_TOKEN_ORDER), ("seq", B.DEV_BAD_TOKEN), ("page", B.DEV_BAD_PAGE)])
def test_append_channels_bad_ones_raise_the_status_beside_others(what, bit):
    # Channel by channel: blocks start and leave while others raise the status word, looking for tokens across padding.
    n = 20000
    c = Case([n], 4, 2, 64, 16)
    kb = torch.zeros(c.k.shape[0], 2, 2, 64, dtype=BF, device="cuda")
    kv = PagedKV(4, 2, 64, 16, max_seqs=1, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    seq[1::3] = -1
    table = c.table.clone()
    if what == "order":
        pos[9000::3000] = 2
    elif what == "seq":
        seq[9000::3000] = 1
    else:
        table[0, 700::300] = c.k.shape[0]
    x = torch.zeros(n, 2, 64, dtype=BF, device="cuda")
    kv.append(x, x, table, seq, pos, q=torch.zeros(n, 4, 64, dtype=BF, device="cuda"), rope=rope_table(n, 10))
    assert kv.status_value() & bit


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 8, 64, 1024])
@pytest.mark.parametrize("length,step", [(100, 3), (100, 33), (2000, 700), (9000, 2), (30000, 7)])
def test_append_between_cached_positions(dtype, page, length, step):
    # Every step-th position is written anew, with padding here and there: the others keep their keys, and the bounds of a
    # page are those of both up to its last new key.
    hq, hkv, d = 8, 2, 64
    c = Case([length, 50], hq, hkv, d, page, dtype)
    kb = torch.zeros(c.k.shape[0], hkv, 2, d, dtype=dtype, device="cuda")
    kv = PagedKV(hq, hkv, d, page, max_seqs=2, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    pos = torch.arange(1, length, step, dtype=torch.int32)
    seq = torch.zeros_like(pos)
    gap = torch.full((40,), -1, dtype=torch.int32)
    at = len(pos) // 2
    pos, seq = torch.cat((pos[:at], gap, pos[at:])).cuda(), torch.cat((seq[:at], gap, seq[at:])).cuda()
    new = torch.randn(len(pos), 2, hkv, d, device="cuda").to(dtype)
    before_k, before_v = c.k.clone(), c.v.clone()
    kv.append(new[:, 0], new[:, 1], c.table, seq, pos)
    kv.check_status()
    real = seq >= 0
    p = pos[real].long()
    where = c.table[0, p // page].long()
    before_k[where, :, p % page] = new[real, 0]
    before_v[where, :, p % page] = new[real, 1]
    assert torch.equal(c.k.nan_to_num(77.0), before_k.nan_to_num(77.0))
    assert torch.equal(c.v.nan_to_num(77.0), before_v.nan_to_num(77.0))
    want = torch.zeros_like(kb)
    last = {}
    for e, off in zip((p // page).tolist(), (p % page).tolist()):
        last[e] = off
    for e, off in last.items():
        keys = before_k[c.table[0, e].long(), :, : off + 1]
        want[c.table[0, e].long(), :, 0], want[c.table[0, e].long(), :, 1] = keys.amin(1), keys.amax(1)
    assert torch.equal(kb, want)


def test_append_follows_a_sequence_that_was_cut_back():
    # Ten positions written, five of them given up, one written anew: the bounds are those of the six that count.
    c = run_append([10], [10], 4, 2, 64, 16, BF, 64, False)
    kb = torch.zeros(c.k.shape[0], 2, 2, 64, dtype=BF, device="cuda")
    kv = PagedKV(4, 2, 64, 16, max_seqs=1, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.randn(1, 2, 64, device="cuda").to(BF)
    kv.append(new, new, c.table, one, one + 5)
    p = int(c.table[0, 0])
    assert torch.equal(c.k[p, :, 5], new[0])
    assert torch.equal(kb[p, :, 0], c.k[p, :, :6].amin(1)) and torch.equal(kb[p, :, 1], c.k[p, :, :6].amax(1))


@pytest.mark.parametrize("seq,pos,bit", [
    ([0, 0], [3, 3], B.DEV_TOKEN_ORDER), ([0, 0], [4, 3], B.DEV_TOKEN_ORDER), ([1, 0], [0, 0], B.DEV_TOKEN_ORDER),
    ([0, -1, -1, 0], [3, 0, 0, 3], B.DEV_TOKEN_ORDER), ([2, 3], [0, 0], B.DEV_BAD_TOKEN), ([0, 1], [-1, 0], B.DEV_BAD_TOKEN),
    ([0, 1], [0, 64], B.DEV_BAD_TOKEN), ([0, 1], [0, 1 << 30], B.DEV_BAD_TOKEN), ([0, 1], [0, 50], B.DEV_BAD_TOKEN),
    ([0, 2], [0, 20], B.DEV_BAD_PAGE)])
def test_append_bad_tokens_raise_the_status(seq, pos, bit):
    # Three sequences of up to 64 positions, a rope table of 50; sequence 2 has no second page.
    c = Case([40, 64, 10], 4, 2, 64, 16)
    kb = torch.zeros(c.k.shape[0], 2, 2, 64, dtype=BF, device="cuda")
    kv = PagedKV(4, 2, 64, 16, max_seqs=3, max_pages=4, k_cache=c.k, v_cache=c.v, k_bounds=kb)
    n = len(seq)
    x = torch.zeros(n, 2, 64, dtype=BF, device="cuda")
    t = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    kv.append(x, x, c.table, t(seq), t(pos), q=torch.zeros(n, 4, 64, dtype=BF, device="cuda"),
              rope=rope_table(50, 64))
    assert kv.status_value() == bit


# ------------------------------------------------------------------ select
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d,page,n_select,first,last", [
    (32, 4, 128, 16, 12, 1, 1), (8, 8, 64, 8, 5, 0, 0), (6, 2, 80, 4, 30, 2, 3), (1, 1, 8, 1, 100, 1, 1), (16, 1, 96, 16, 1, 0, 1),
    (8, 2, 64, 16, 3, 2, 4), (40, 1, 24, 16, 200, 1, 1)])
def test_select(dtype, hq, hkv, d, page, n_select, first, last):
    c = Case([0, 1, 17, 500, 16, 1203], hq, hkv, d, page, dtype, seed=d)
    # Bounds of all pages, NaN where there is no key (nan-ignoring minima), zero for unused pages.
    lo, hi = c.k.float().nan_to_num(nan=float("inf")).amin(2), c.k.float().nan_to_num(nan=-float("inf")).amax(2)
    kb = torch.stack((lo, hi), 2).clamp(-50, 50).to(dtype).contiguous()
    kv = PagedKV(hq, hkv, d, page, max_seqs=6, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    pages = kv.select(c.q, c.table, c.lens, n_select, keep_first=first, keep_last=last)
    kv.check_status()
    want = OP.select(f64(c.q), f64(kb), c.table.cpu().numpy(), c.lens_l, page, n_select, first, last)
    assert np.array_equal(pages.cpu().numpy(), want)
    o, lse = kv.decode(c.q, c.table, c.lens, pages=pages)
    kv.check_status()
    c.check(o, lse, c.oracle(pages=want))


@pytest.mark.parametrize("count,n_select", [(5000, 64), (5000, 4999), (300, 7), (20000, 300), (257, 256)])
def test_select_ties_and_long_rows(count, n_select):
    # Small whole numbers: many equal scores, in every arithmetic; ties go to the lower page.
    g = torch.Generator().manual_seed(count)
    d, hkv, hq = 8, 2, 4
    kb = torch.randint(-2, 3, (count + 1, hkv, 2, d), generator=g).float().sort(2).values.to(BF).cuda()
    k = torch.zeros(count + 1, hkv, 1, d, dtype=BF, device="cuda")
    q = torch.randint(-1, 2, (2, hq, d), generator=g).to(BF).cuda()
    table = torch.stack([torch.randperm(count + 1, generator=g)[:count] for _ in range(2)]).to(torch.int32).cuda()
    lens = torch.tensor([count, count // 3], dtype=torch.int32).cuda()
    kv = PagedKV(hq, hkv, d, 1, max_seqs=2, max_pages=count, k_cache=k, v_cache=k, k_bounds=kb)
    got = kv.select(q, table, lens, n_select, keep_first=2, keep_last=1).cpu().numpy()
    kv.check_status()
    qn, bn, tn = f64(q), f64(kb), table.cpu().numpy()
    for b in range(2):
        n = int(lens[b])
        for h in range(hkv):
            lo, hi = bn[tn[b, :n], h, 0], bn[tn[b, :n], h, 1]
            s = sum(np.maximum(qn[b, x] * lo, qn[b, x] * hi).sum(1) for x in (2 * h, 2 * h + 1))
            s[:2], s[n - 1] = np.inf, np.inf
            want = np.sort(np.argsort(-s, kind="stable")[:n_select])
            assert got[b, h, :len(want)].tolist() == want.tolist() and (got[b, h, len(want):] == -1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_seqs,count,n_select", [(100, 6000, 50), (1, 131072, 1000), (90, 700, 699), (2, 49152, 900),
                                                   (80, 24000, 30), (1, 49153, 64)])
def test_select_many_rows_and_the_longest(dtype, n_seqs, count, n_select):
    g = torch.Generator().manual_seed(count)
    d, hkv, hq = 16, 2, 6
    kb = torch.randn(count + 1, hkv, 2, d, generator=g).sort(2).values.to(dtype).cuda()
    k = torch.zeros(count + 1, hkv, 1, d, dtype=dtype, device="cuda")
    q = torch.randn(n_seqs, hq, d, generator=g).to(dtype).cuda()
    table = torch.stack([torch.randperm(count + 1, generator=g)[:count] for _ in range(n_seqs)]).to(torch.int32).cuda()
    lens = torch.randint(0, count + 1, (n_seqs,), generator=g, dtype=torch.int32)
    lens[0] = count
    kv = PagedKV(hq, hkv, d, 1, max_seqs=n_seqs, max_pages=count, k_cache=k, v_cache=torch.zeros_like(k), k_bounds=kb)
    got = kv.select(q, table, lens.cuda(), n_select, keep_first=1, keep_last=2).cpu().numpy()
    kv.check_status()
    qn, bn, tn = f64(q), f64(kb), table.cpu().numpy()
    for b in range(n_seqs):
        n = int(lens[b])
        for h in range(hkv):
            qg = qn[b, 3 * h : 3 * h + 3]
            up, down = np.maximum(qg, 0).sum(0), np.minimum(qg, 0).sum(0)
            s = bn[tn[b, :n], h, 1] @ up + bn[tn[b, :n], h, 0] @ down
            s[:1], s[max(n - 2, 0):] = np.inf, np.inf
            want = np.sort(np.argsort(-s, kind="stable")[:n_select])
            assert got[b, h, :len(want)].tolist() == want.tolist() and (got[b, h, len(want):] == -1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_most_sequences(dtype):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 40, B.PAGED_MAX_SEQS).tolist()
    run_append([n + 1 for n in lens], [1] * len(lens), 4, 2, 16, 4, dtype, 16, False)
    c = Case(lens, 4, 2, 16, 4, dtype)
    c.check(*c.kv.decode(c.q, c.table, c.lens), c.oracle())
    c.kv.check_status()
    kb = torch.randn(c.k.shape[0], 2, 2, 16, generator=torch.Generator().manual_seed(2)).sort(2).values.to(dtype).cuda()
    kv = PagedKV(4, 2, 16, 4, max_seqs=len(lens), max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    pages = kv.select(c.q, c.table, c.lens, 3)
    want = OP.select(f64(c.q), f64(kb), c.table.cpu().numpy(), lens, 4, 3, 1, 1)
    assert np.array_equal(pages.cpu().numpy(), want)
    c.check(*kv.decode(c.q, c.table, c.lens, pages=pages), c.oracle(pages=want))
    kv.check_status()


def test_select_far_scores_and_nan():
    # Scores over the whole range of exponents; a NaN score ranks below all. The score is sum_i a_i kmax_i + b_i kmin_i
    # with b_i = 0 here, so an infinite bound gives 0 * inf = NaN too; pages of equal (lowest) rank go by their index.
    n = 40
    kb = torch.zeros(n, 1, 2, 8, dtype=F32, device="cuda")
    kb[:, 0, :, 0] = torch.tensor([(-1.0) ** i * 2.0 ** (i - 20) for i in range(n)])[:, None].cuda()
    kb[3, 0, :, 0] = float("nan")
    kb[5, 0, :, 0] = float("-inf")
    kb[6, 0, :, 0] = float("inf")
    k = torch.zeros(n, 1, 1, 8, dtype=F32, device="cuda")
    kv = PagedKV(1, 1, 8, 1, max_seqs=1, max_pages=n, k_cache=k, v_cache=k, k_bounds=kb)
    q = torch.zeros(1, 1, 8, device="cuda")
    q[0, 0, 0] = 1.0
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    order = sorted((i for i in range(n) if i not in (3, 5, 6)), key=lambda i: -((-1.0) ** i * 2.0 ** (i - 20)))
    order = order + [3, 5, 6]
    for m in (1, 2, 20, 37, 38, 39, 40):
        got = kv.select(q, table, lens, m, keep_first=0, keep_last=0)[0, 0].tolist()
        assert got == sorted(order[:m]), m


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e6])
def test_select_bounds_of_kept_pages_do_not_count(dtype, value):
    # Pages that are taken anyway hold what makes a score say nothing: the others are chosen as without them, and from their
    # float32 scores (the second word of a page's score is set for one page of a warp's share only; scored again in float64,
    # all of them hold other things).
    count, d, hkv, hq, n_select = 4096, 128, 2, 8, 64
    g = torch.Generator().manual_seed(5)
    kb = torch.randn(count, hkv, 2, d, generator=g).sort(2).values.to(dtype).cuda()
    table = torch.randperm(count, generator=g).to(torch.int32)[None].cuda()
    q = torch.randn(1, hq, d, generator=g).to(dtype).cuda()
    up, down = (x.sum(1) for x in (lambda y: (np.maximum(y, 0), np.minimum(y, 0)))(f64(q)[0].reshape(hkv, -1, d)))
    bn = f64(kb)[table[0].cpu().numpy()]
    for p in (0, 1, count - 3, count - 2, count - 1):
        kb[table[0, p].long()] = value
    k = torch.zeros(count, hkv, 1, d, dtype=dtype, device="cuda")
    paged = B.make_paged(hq, hkv, d, 1, count, count, k.stride()[:3], dtype=dtype)
    ws = torch.zeros(B.splitkv_paged_select_workspace_size(paged, 1) // 4, dtype=torch.int32, device="cuda")
    pages = torch.empty(1, hkv, n_select, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.splitkv_paged_select(paged, 1, q, hq * d, kb, table, torch.tensor([count], dtype=torch.int32).cuda(), n_select, 2, 3,
                           pages, status, ws)
    assert int(status) == 0
    for h in range(hkv):
        s = bn[:, h, 1] @ up[h] + bn[:, h, 0] @ down[h]
        s[:2], s[-3:] = np.inf, np.inf
        assert pages[0, h].tolist() == sorted(np.argsort(-s, kind="stable")[:n_select].tolist())
    assert int((ws.view(hkv, count, 2)[:, :, 1] != 0).sum()) <= hkv * count // 4


def test_select_bad_pages_and_lengths():
    c = Case([64, 64], 4, 2, 64, 16)
    kb = torch.zeros(c.k.shape[0], 2, 2, 64, dtype=BF, device="cuda")
    kv = PagedKV(4, 2, 64, 16, max_seqs=2, max_pages=4, k_cache=c.k, v_cache=c.v, k_bounds=kb)
    table = c.table.clone()
    table[1, 2] = kb.shape[0]
    kv.select(c.q, table, c.lens, 2)
    assert kv.status_value() == B.DEV_BAD_PAGE
    kv.status.zero_()
    kv.select(c.q, c.table, torch.tensor([64, 65], dtype=torch.int32).cuda(), 2)
    assert kv.status_value() == B.DEV_BAD_LENGTH


# ------------------------------------------------------------------ streams, graphs, a run of all of them
def test_streams_share_one_object():
    # Calls that alternate between streams use the same scratch in turn: the same results, bit for bit.
    c = Case([8000, 4000, 100], 32, 4, 128, 16)
    want = [x.clone() for x in c.kv.decode(c.q, c.table, c.lens)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(30):
        if i % 2:
            with torch.cuda.stream(streams[i % 3]):
                got.append(c.kv.decode(c.q, c.table, c.lens))
        else:
            got.append(c.kv.decode(c.q, c.table, c.lens, stream=streams[i % 3]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for pair in got for x, y in zip(pair, want))
    raw = c.kv.decode(c.q, c.table, c.lens, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw[0], want[0])


def test_calls_see_what_the_kernel_before_them_wrote():
    # Lengths, tokens and queries change right before each call, without a wait: the results are those of calls made apart.
    c = Case([4000, 3000, 9], 8, 2, 64, 16)
    kb = torch.randn(c.k.shape[0], 2, 2, 64, device="cuda").sort(2).values.to(BF)
    kv = PagedKV(8, 2, 64, 16, max_seqs=3, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    n = 6000  # with queries: two launches
    many_q = torch.randn(n, 8, 64, device="cuda").to(BF)
    inputs = []
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        inputs.append(dict(lens=torch.tensor([4000 - 700 * i, 100 + 900 * i, i], dtype=torch.int32),
                           pos=torch.cat((torch.arange(3500) + 10 * i, torch.arange(2500) + 50 * i)).to(torch.int32),
                           q=torch.randn(3, 8, 64, generator=g).to(BF), x=torch.randn(n, 2, 64, generator=g).to(BF)))
    inputs = [{k: v.cuda() for k, v in x.items()} for x in inputs]
    seq = torch.cat((torch.zeros(3500), torch.ones(2500))).to(torch.int32).cuda()
    now = {k: v.clone() for k, v in inputs[0].items()}
    state = [c.k, c.v, kb]
    start = [t.clone() for t in state]

    def step(x, apart):
        got = []
        for call in (lambda: kv.append(now["x"], now["x"], c.table, seq, now["pos"], q=many_q),
                     lambda: got.append(kv.select(now["q"], c.table, now["lens"], 30)),
                     lambda: got.extend(kv.decode(now["q"], c.table, now["lens"])),
                     lambda: got.extend(kv.decode(now["q"], c.table, now["lens"], pages=got[0]))):
            for k, v in now.items():
                v.copy_(x[k])
            if apart:
                torch.cuda.synchronize()
            call()
            if apart:
                torch.cuda.synchronize()
        return got + [t.clone() for t in state]

    def run(apart):
        for t, s in zip(state, start):
            t.copy_(s)
        return [step(inputs[i % 4], apart) for i in range(24)]

    want, got = run(True), run(False)
    kv.check_status()
    for w, g in zip(want, got):
        assert all(torch.equal(x.nan_to_num(77.0), y.nan_to_num(77.0)) for x, y in zip(w, g))


def _ranges(tensors):
    return [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in tensors]


def _meet(ranges, tensors):
    return any(p < q + m and q < p + n for p, n in ranges for q, m in _ranges(tensors))


@pytest.mark.parametrize("call", ["decode", "select", "append"])
def test_a_dropped_object_keeps_its_memory_until_its_calls_are_done(call):
    # Work of a call on another stream than the memory's own is still waiting there when the last reference goes.
    c = Case([3000], 8, 2, 64, 16)
    kv = PagedKV(8, 2, 64, 16, max_seqs=1, max_pages=c.table.shape[1], n_pages=c.k.shape[0], bounds=True)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    for t in (kv.k_cache, kv.v_cache, kv.k_bounds):
        t.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = _ranges([kv.k_cache, kv.v_cache, kv.k_bounds, kv._ws])
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # 0.2 s
        if call == "decode":
            kv.decode(c.q, c.table, c.lens)
        elif call == "select":
            kv.select(c.q, c.table, c.lens, 5)
        else:
            kv.append(x, x, c.table, one, one)
    del kv
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in held]
    waiting = not side.query()
    met = _meet(held, others)
    torch.cuda.synchronize()
    assert waiting and not met
    del others
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in held]
    assert _meet(held, again)  # then it is given back


@pytest.mark.parametrize("raw", [False, True])
def test_tensors_of_a_call_on_a_given_stream_may_be_dropped(raw):
    c = Case([3000], 8, 2, 64, 16)
    kb = torch.zeros(c.k.shape[0], 2, 2, 64, dtype=BF, device="cuda")
    kv = PagedKV(8, 2, 64, 16, max_seqs=1, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    rope = rope_table(16, 64)
    pages = kv.select(c.q, c.table, c.lens, 5)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else side

    def fresh(t):
        return t.clone(memory_format=torch.contiguous_format)

    for call, given in ((lambda a: kv.decode(*a, stream=handle), (c.q, c.table, c.lens, pages)),
                        (lambda a: kv.decode(*a[:3], o=a[3], lse=a[4], stream=handle),
                         (c.q, c.table, c.lens, torch.empty_like(c.q), torch.empty(1, 8, device="cuda"))),
                        (lambda a: kv.select(*a, 5, stream=handle), (c.q, c.table, c.lens)),
                        (lambda a: kv.append(*a[:5], q=a[5], rope=a[6], stream=handle), (x, x, c.table, one, one, c.q, rope))):
        given = [fresh(t) for t in given]
        torch.cuda.synchronize()
        held, sizes = _ranges(given), [t.untyped_storage().nbytes() for t in given]
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)  # 0.2 s
        got = call(given)
        given.clear()
        others = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        waiting, met = not side.query(), _meet(held, others)
        torch.cuda.synchronize()
        assert waiting and not met
        del got, others


def test_a_graph_outlives_the_object_it_was_captured_from():
    # Caches, bounds and outputs are kept, the object is not; what it held is somebody else's by the time of the replay.
    c = Case([3000, 40], 8, 2, 64, 16)
    kb = torch.randn(c.k.shape[0], 2, 2, 64, device="cuda").sort(2).values.to(BF)
    kv = PagedKV(8, 2, 64, 16, max_seqs=2, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    want = [t.clone() for t in (*kv.decode(c.q, c.table, c.lens), kv.select(c.q, c.table, c.lens, 5))]
    got = [torch.zeros_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.decode(c.q, c.table, c.lens, o=got[0], lse=got[1])
        kv.select(c.q, c.table, c.lens, 5, pages=got[2])
    size = kv._ws.numel()
    del kv
    gc.collect()
    taken = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in [size // 4 + 4, size // 4] + [4] * 600]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(bool((t == -1).all()) for t in taken)


def test_status_words_are_apart():
    c = Case([64], 4, 2, 64, 16)
    kvs = [PagedKV(4, 2, 64, 16, max_seqs=1, max_pages=4, k_cache=c.k, v_cache=c.v) for _ in range(140)]
    assert len({kv.status.data_ptr() for kv in kvs}) == len(kvs)
    kvs[77].decode(c.q, c.table, c.lens + 1)
    assert [kv.status_value() for kv in kvs] == [B.DEV_BAD_LENGTH if i == 77 else 0 for i in range(140)]


def test_graphs_follow_their_inputs_and_share_nothing():
    # Two graphs of one object, replayed side by side with eager calls between: each keeps its results.
    c = Case([6000, 3000], 32, 4, 128, 16)
    lens = [c.lens.clone(), c.lens.clone()]
    graphs, outs = [], []
    for i in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.kv.decode(c.q, c.table, lens[i])  # warm-up
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(c.kv.decode(c.q, c.table, lens[i]))
        graphs.append((g, s))
    lens[1].copy_(torch.tensor([17, 2999], dtype=torch.int32))
    torch.cuda.synchronize()
    refs = [c.oracle(), c.oracle(lens=[17, 2999])]
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager = c.kv.decode(c.q, c.table, c.lens)
    torch.cuda.synchronize()
    c.check(*outs[0], refs[0])
    c.check(*outs[1], refs[1])
    c.check(*eager, refs[0])
    c.kv.check_status()


def test_a_graph_of_several_streams():
    # One capture: an append, then attention over all keys and over chosen pages side by side, then the next append.
    c = Case([2000, 700, 1], 8, 2, 64, 16)
    kb = torch.randn(c.k.shape[0], 2, 2, 64, device="cuda").sort(2).values.to(BF)
    kv = PagedKV(8, 2, 64, 16, max_seqs=3, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    seq = torch.arange(3, dtype=torch.int32, device="cuda")
    new = torch.randn(4, 3, 2, 64, device="cuda").to(BF)
    side = torch.cuda.Stream()

    def run(fork):
        got = []
        for x in new:
            main = torch.cuda.current_stream()
            kv.append(x, x, c.table, seq, c.lens - 1)
            if fork:
                side.wait_stream(main)
            with torch.cuda.stream(side if fork else main):
                pages = kv.select(c.q, c.table, c.lens, 9)
                sparse = kv.decode(c.q, c.table, c.lens, pages=pages)
            got += [*kv.decode(c.q, c.table, c.lens), pages, *sparse]
            if fork:
                main.wait_stream(side)
        return got

    want = [t.clone() for t in run(False)]
    state = [t.clone() for t in (c.k, c.v, kb)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(True)
    for t in (c.k[c.table[0, 0].long()], c.v[c.table[0, 0].long()]):
        assert not t.isnan().any()
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x.nan_to_num(77.0), y.nan_to_num(77.0)) for x, y in zip((c.k, c.v, kb), state))
    kv.check_status()


def test_threads_share_one_object():
    # Each thread on a stream of its own: decode, select and decode over the list, all on one object.
    c = Case([9000, 50, 0, 700], 8, 2, 64, 16)
    kb = torch.randn(c.k.shape[0], 2, 2, 64, device="cuda").sort(2).values.to(BF)
    kv = PagedKV(8, 2, 64, 16, max_seqs=4, max_pages=c.table.shape[1], k_cache=c.k, v_cache=c.v, k_bounds=kb)
    o, lse = kv.decode(c.q, c.table, c.lens)
    pages = kv.select(c.q, c.table, c.lens, 20)
    so, slse = kv.decode(c.q, c.table, c.lens, pages=pages)
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(40):
                a = kv.decode(c.q, c.table, c.lens)
                p = kv.select(c.q, c.table, c.lens, 20)
                b = kv.decode(c.q, c.table, c.lens, pages=p)
                if not all(torch.equal(x, y) for x, y in zip((*a, p, *b), (o, lse, pages, so, slse))):
                    wrong.append(1)
        stream.synchronize()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    kv.check_status()


def test_an_eager_call_beside_a_capture_stays_out_of_it():
    # The object's last eager call was on the stream that is being captured: an eager call on another stream runs at once.
    c = Case([3000, 40], 8, 2, 64, 16)
    want = [t.clone() for t in c.kv.decode(c.q, c.table, c.lens)]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.kv.decode(c.q, c.table, c.lens)  # warm-up
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
        captured = c.kv.decode(c.q, c.table, c.lens)
        c.kv.decode(c.q, c.table, c.lens, o=o, lse=lse, stream=t)
        assert not c.kv._capturing(t)
        t.synchronize()
        with torch.cuda.stream(t):
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
        c.kv.decode(c.q, c.table, c.lens, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(captured[0], want[0]) and torch.equal(captured[1], want[1]) and not o.any()
    c.kv.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_serving_run(dtype):
    """Prompts appended (in two pieces), then tokens one by one as one captured step: append, select, sparse and full
    attention. At each step the attention equals the oracle's over the keys and values appended so far."""
    hq, hkv, d, page, n, steps, n_select = 8, 2, 64, 16, 3, 6, 4
    prompts = [37, 5, 90]
    g = torch.Generator().manual_seed(11)
    width = -(-(max(prompts) + steps) // page)
    kv = PagedKV(hq, hkv, d, page, max_seqs=n, max_pages=width, n_pages=n * width + 2, dtype=dtype, bounds=True)
    kv.k_cache.fill_(float("nan"))
    kv.v_cache.fill_(float("nan"))
    kv.k_bounds.fill_(float("nan"))
    table = torch.randperm(n * width + 2, generator=g)[:n * width].view(n, width).to(torch.int32).cuda()
    rope = rope_table(width * page, d)
    all_qkv = [torch.randn(p + steps, hq + 2 * hkv, d, generator=g).to(dtype) for p in prompts]

    def split(x):
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    for lo, hi in ((0.0, 0.4), (0.4, 1.0)):
        part = [(b, int(p * lo), int(p * hi)) for b, p in enumerate(prompts)]
        x = torch.cat([all_qkv[b][s:e] for b, s, e in part]).cuda()
        seq = torch.tensor([b for b, s, e in part for _ in range(s, e)], dtype=torch.int32).cuda()
        pos = torch.tensor([i for b, s, e in part for i in range(s, e)], dtype=torch.int32).cuda()
        q, k, v = split(x)
        kv.append(k, v, table, seq, pos, q=q, rope=rope)
    # One step, captured: its inputs are buffers that the loop refills.
    x = torch.zeros(n, hq + 2 * hkv, d, dtype=dtype, device="cuda")
    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    seq = torch.arange(n, dtype=torch.int32, device="cuda")

    def step():
        q, k, v = split(x)
        q = kv.append(k, v, table, seq, lens, q=q, rope=rope)
        lens.add_(1)
        pages = kv.select(q, table, lens, n_select)
        return q, pages, kv.decode(q, table, lens, pages=pages), kv.decode(q, table, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        x.copy_(torch.stack([all_qkv[b][prompts[b]] for b in range(n)]).cuda())
        step()
        lens.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        q, pages, sparse, full = step()
    like_case = type("C", (), dict(dtype=dtype, d=d, lens_l=[max(prompts) + steps]))
    for t in range(steps):
        x.copy_(torch.stack([all_qkv[b][prompts[b] + t] for b in range(n)]).cuda())
        graph.replay()
        torch.cuda.synchronize()
        kv.check_status()
        now = [p + t + 1 for p in prompts]
        assert lens.tolist() == now
        tn, kn, vn = table.cpu().numpy(), f64(kv.k_cache), f64(kv.v_cache)
        for b in range(n):  # the cache holds the rotated keys
            want = np.stack([OP.rope(f64(split(all_qkv[b])[1][i]), f64(rope)[i, :d // 2], f64(rope)[i, d // 2:], False)
                             for i in range(now[b])], 1)
            got = np.stack([OP.keys_of(kn, tn[b], h, now[b]) for h in range(hkv)])
            assert np.abs(got - want).max() <= half_step(dtype) * np.abs(want).max() + 1e-5
        want = OP.select(f64(q), f64(kv.k_bounds), tn, now, page, n_select, 1, 1)
        assert np.array_equal(pages.cpu().numpy(), want)
        Case.check(like_case, *full, OP.decode(f64(q), kn, vn, tn, now, 1 / np.sqrt(d)))
        Case.check(like_case, *sparse, OP.decode(f64(q), kn, vn, tn, now, 1 / np.sqrt(d), want))


def test_no_sequences_and_no_tokens():
    c = Case([10], 4, 2, 64, 16)
    o, lse = c.kv.decode(c.q[:0], c.table[:0], c.lens[:0])
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    z = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    before = c.k.clone()
    assert c.kv.append(z, z, c.table, i, i) is None
    assert torch.equal(before.nan_to_num(), c.k.nan_to_num())
    c.kv.check_status()
