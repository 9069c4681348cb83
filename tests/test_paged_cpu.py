"""The paged-cache operators without a GPU: the oracle against explicit formulas, and every refusal before a launch."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import paged as OP

B = pytest.importorskip("split_kv_lse_splitkv_b200.binding", reason="libsplitkv.so not built")
from split_kv_lse_splitkv_b200.paged import PagedKV, rope_table  # noqa: E402


# ------------------------------------------------------------------ the oracle
def test_oracle_decode_is_softmax_attention(rng):
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((5, 2, 4, 8)), rng.standard_normal((5, 2, 4, 8))
    table = np.array([[3, 1, 0], [4, 2, 2]])
    o, lse, _, _ = OP.decode(q, k, v, table, [9, 0], 0.3)
    rows_k = np.concatenate([k[3], k[1], k[0]], 1)[:, :9]
    rows_v = np.concatenate([v[3], v[1], v[0]], 1)[:, :9]
    for h in range(4):
        s = 0.3 * rows_k[h // 2] @ q[0, h]
        p = np.exp(s) / np.exp(s).sum()
        assert np.allclose(o[0, h], p @ rows_v[h // 2], rtol=1e-12) and np.isclose(lse[0, h], np.log(np.exp(s).sum()))
    assert (o[1] == 0).all() and (lse[1] == -np.inf).all()
    # All pages listed: the same; the parts over two lists join to the whole.
    both = OP.decode(q[:1], k, v, table[:1], [9], 0.3, pages=np.array([[[0, 1, 2]] * 2]))
    assert np.allclose(both[0], o[:1]) and np.allclose(both[1], lse[:1])
    parts = [OP.decode(q[:1], k, v, table[:1], [9], 0.3, pages=np.array([[x] * 2])) for x in ([0, 2], [1])]
    L = np.logaddexp(parts[0][1], parts[1][1])
    joined = sum(np.exp(x[1] - L)[..., None] * x[0] for x in parts)
    assert np.allclose(L, lse[:1]) and np.allclose(joined, o[:1])


def test_oracle_rope_is_a_rotation(rng):
    # The product of two rotated rows depends on the distance of their positions only, in either pairing.
    table = rope_table(40, 6, base=100.0, device="cpu").double().numpy()
    q, k = rng.standard_normal((1, 10)), rng.standard_normal((1, 10))
    for pairs in (False, True):
        dots = [(OP.rope(q, table[i + 7, :3], table[i + 7, 3:], pairs) @ OP.rope(k, table[i, :3], table[i, 3:], pairs).T)
                for i in (0, 11, 32)]
        assert np.allclose(dots, dots[0], atol=1e-6)  # the table is float32
        assert np.allclose(OP.rope(q, table[0, :3], table[0, 3:], pairs), q)


def test_oracle_scores_bound_every_key(rng):
    q, k = rng.standard_normal((6, 5)), rng.standard_normal((7, 2, 4, 5))
    bounds = np.stack([k.min(2), k.max(2)], 2)
    s = OP.scores(q, bounds, np.arange(7), 1, 7)
    real = np.einsum("hd,ptd->pt", q[3:], k[:, 1])
    assert (real.max(1) <= s + 1e-12).all()
    # The linear form that the kernels use.
    up, down = np.maximum(q[3:], 0).sum(0), np.minimum(q[3:], 0).sum(0)
    assert np.allclose(s, bounds[:, 1, 1] @ up + bounds[:, 1, 0] @ down)


def test_oracle_select_ties_and_kept_pages():
    q = np.ones((1, 1, 2))
    bounds = np.zeros((6, 1, 2, 2))
    bounds[:, 0, 1] = np.array([0, 5, 5, 1, 5, 0])[:, None]
    table = np.arange(6)[None]
    assert OP.select(q, bounds, table, [12], 2, 2, 0, 0)[0, 0].tolist() == [1, 2]
    assert OP.select(q, bounds, table, [11], 2, 4, 1, 1)[0, 0].tolist() == [0, 1, 2, 5]
    assert OP.select(q, bounds, table, [11], 2, 2, 2, 2)[0, 0].tolist() == [0, 1]
    assert OP.select(q, bounds, table, [3], 2, 4, 1, 1)[0, 0].tolist() == [0, 1, -1, -1]
    assert OP.select(q, bounds, table, [0], 2, 2, 1, 1)[0, 0].tolist() == [-1, -1]


def test_rope_table():
    t = rope_table(5, 8, base=1000.0, device="cpu")
    assert t.shape == (5, 8) and t.dtype == torch.float32
    ang = 3 * 1000.0 ** (-np.arange(4) / 4)
    assert np.allclose(t[3].numpy(), np.concatenate([np.cos(ang), np.sin(ang)]), atol=1e-7)
    # A far position: the angle itself is right to float64, not to float32.
    far = rope_table(1 << 20, 2, device="cpu")[-1].numpy()
    assert abs(far[0] - np.cos(float((1 << 20) - 1))) < 1e-7
    for bad in ((0, 8), (4, 7), (4, 0)):
        with pytest.raises(B.SplitKVError):
            rope_table(*bad, device="cpu")


# ------------------------------------------------------------------ the C ABI's refusals
def desc(**kw):
    a = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_pages=4,
             strides=(2 * 16 * 64, 16 * 64, 64), dtype=torch.bfloat16)
    a.update(kw)
    return B.make_paged(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=7), B.EINVAL),
    (dict(n_kv_heads=0), B.EINVAL),
    (dict(head_dim=60), B.EUNSUPPORTED),                                   # not a multiple of 16 bytes
    (dict(head_dim=136, strides=(2 * 16 * 136, 16 * 136, 136)), B.EUNSUPPORTED),
    (dict(page_size=12), B.EUNSUPPORTED),                                  # not a power of two
    (dict(page_size=2048), B.EUNSUPPORTED),
    (dict(page_size=0), B.EINVAL),
    (dict(n_pages=0), B.EINVAL),
    (dict(max_pages=0), B.EINVAL),
    (dict(max_pages=1 << 28), B.EUNSUPPORTED),                             # a sequence of 2^32 positions
    (dict(page_size=1, max_pages=(1 << 31) - 1, n_kv_heads=1), B.EUNSUPPORTED),  # rounded up to a tile: 2^31 positions
    (dict(table_stride=3), B.EINVAL),
    (dict(scale=0.0), B.EINVAL),
    (dict(scale=float("nan")), B.EINVAL),
    (dict(scale=float("inf")), B.EINVAL),
    (dict(strides=(2 * 16 * 64, 16 * 64, 60)), B.EINVAL),                  # rows overlap
    (dict(strides=(2 * 16 * 64, 15 * 64, 64)), B.EINVAL),                  # heads overlap
    (dict(strides=(16 * 64, 16 * 64, 64)), B.EINVAL),                      # pages overlap
    (dict(strides=(2 * 16 * 64 + 4, 16 * 64, 64)), B.EINVAL),              # not a multiple of 16 bytes
    (dict(strides=(0, 16 * 64, 64)), B.EINVAL),
])
def test_bad_descriptions_are_refused(kw, code):
    fake = torch.empty(64, dtype=torch.int32)
    p = desc(**kw)
    assert B.splitkv_paged_workspace_size(p, 4) == 0
    with pytest.raises(B.SplitKVError) as e:
        B.splitkv_paged_decode(p, 4, fake, 512, fake, fake, fake, fake, None, 0, fake, fake, fake, fake, stream=0)
    assert e.value.code == code


def test_work_that_a_call_may_hold():
    # 4096 sequences of up to a million positions at 8 kv heads; and what one sequence alone is too much for.
    many = desc(n_q_heads=8, n_kv_heads=8, page_size=64, max_pages=16384, strides=(8 * 64 * 64, 64 * 64, 64))
    assert B.splitkv_paged_workspace_size(many, B.PAGED_MAX_SEQS) > 0
    kv = make(n_kv_heads=8, page_size=64, max_pages=16384, max_seqs=B.PAGED_MAX_SEQS)
    assert kv.max_seqs == B.PAGED_MAX_SEQS
    f = torch.empty(64, dtype=torch.int32)
    for pages, heads, fits in ((1 << 21, 16, True), (1 << 21, 17, False), (1 << 14, 2048, True), (1 << 14, 2049, False)):
        p = desc(n_q_heads=heads, n_kv_heads=heads, head_dim=8, page_size=1024, max_pages=pages - 3, table_stride=1 << 22,
                 strides=(heads * 1024 * 8, 1024 * 8, 8))
        assert (B.splitkv_paged_workspace_size(p, 1) > 0) == fits
        if not fits:
            with pytest.raises(B.SplitKVError) as e:
                B.splitkv_paged_decode(p, 1, f, 8 * heads, f, f, f, f, None, 0, f, f, f, f, stream=0)
            assert e.value.code == B.EUNSUPPORTED


def test_layouts_that_are_accepted():
    for kw in (dict(), dict(strides=(2 * 16 * 64, 64, 128)),               # [pages, positions, heads, d]
               dict(strides=(16 * 64, 10 * 16 * 64, 64)),                  # [heads, pages, positions, d]
               dict(strides=(2 * 16 * 80, 16 * 80, 80)),                   # rows with a gap
               dict(page_size=1, strides=(128, 64, 8)),                    # one position a page: its stride says nothing
               dict(head_dim=8, strides=(2 * 16 * 8, 16 * 8, 8)),
               dict(dtype=torch.float32, head_dim=12, strides=(2 * 16 * 12, 16 * 12, 12))):
        assert B.splitkv_paged_workspace_size(desc(**kw), 4) > 0
    assert B.splitkv_paged_workspace_size(desc(), 0) > 0
    assert B.splitkv_paged_workspace_size(desc(), -1) == 0
    assert B.splitkv_paged_workspace_size(desc(), B.PAGED_MAX_SEQS + 1) == 0


def test_decode_refusals():
    f = torch.empty(1 << 16, dtype=torch.int32)  # host memory, never dereferenced
    ws = torch.empty(B.splitkv_paged_workspace_size(desc(), 4), dtype=torch.uint8)
    good = dict(q=f, q_stride=512, k_cache=f, v_cache=f, page_table=f, seq_len=f, pages=None, n_select=0, o=f, lse=f,
                status=f, workspace=ws)
    for kw, code in ((dict(q=None), B.EINVAL), (dict(k_cache=None), B.EINVAL), (dict(v_cache=None), B.EINVAL),
                     (dict(page_table=None), B.EINVAL), (dict(seq_len=None), B.EINVAL), (dict(o=None), B.EINVAL),
                     (dict(lse=None), B.EINVAL), (dict(status=None), B.EINVAL), (dict(q=f[1:]), B.EINVAL),
                     (dict(k_cache=f[1:]), B.EINVAL), (dict(v_cache=f[2:]), B.EINVAL), (dict(o=f[3:]), B.EINVAL),
                     (dict(q_stride=504), B.EINVAL), (dict(q_stride=516), B.EINVAL), (dict(q_stride=-512), B.EINVAL),
                     (dict(pages=f, n_select=0), B.EINVAL), (dict(workspace=None), B.ENOSPACE),
                     (dict(workspace=ws[:64]), B.ENOSPACE), (dict(workspace=ws[8:]), B.ENOSPACE)):
        with pytest.raises(B.SplitKVError) as e:
            B.splitkv_paged_decode(desc(), 4, **{**good, **kw}, stream=0)
        assert e.value.code == code, kw
    with pytest.raises(B.SplitKVError) as e:
        B.splitkv_paged_decode(desc(), B.PAGED_MAX_SEQS + 1, **good, stream=0)
    assert e.value.code == B.EUNSUPPORTED
    # No sequence: nothing to do, no tensor is looked at.
    B.splitkv_paged_decode(desc(), 0, **{k: None for k in good} | dict(q_stride=0, n_select=0, status=f), stream=0)


def test_decode_outputs_lie_apart():
    f = [torch.empty(1 << 16, dtype=torch.int32) for _ in range(7)]
    ws = torch.empty(B.splitkv_paged_workspace_size(desc(), 4), dtype=torch.uint8)
    good = dict(q=f[0], q_stride=512, k_cache=f[1], v_cache=f[2], page_table=f[3], seq_len=f[3], pages=None, n_select=0,
                o=f[4], lse=f[5], status=f[6], workspace=ws)
    # q and o: 4 tokens of 1024 bytes; lse: 128 bytes.
    for kw, code in ((dict(o=f[0]), B.EINVAL), (dict(o=f[0][1020:]), B.EINVAL), (dict(lse=f[0][4:]), B.EINVAL),
                     (dict(lse=f[4][1023:]), B.EINVAL), (dict(q=f[4][512:], q_stride=1024), B.EINVAL),
                     (dict(q=f[5][:16]), B.EINVAL), (dict(pages=f[3], n_select=(1 << 29) + 1), B.EUNSUPPORTED)):
        with pytest.raises(B.SplitKVError) as e:
            B.splitkv_paged_decode(desc(), 4, **{**good, **kw}, stream=0)
        assert e.value.code == code, kw


def _apart(call, args, over):
    """Each of `over` = (name, (tensor, first element)) puts one tensor of the call where it may not be."""
    for name, (at, first) in over:
        with pytest.raises(B.SplitKVError) as e:
            call({**args, name: at[first:]})
        assert e.value.code == B.EINVAL, name


def test_decode_writes_apart_from_lists_and_scratch():
    # Elements of 4 bytes: q, o 4 x 256, lse 32, lengths 4, table 16 (rows of 4), pages 4 x 2 x 3.
    f = {k: torch.empty(1 << 16, dtype=torch.int32) for k in ("q", "k_cache", "v_cache", "page_table", "seq_len", "pages", "o", "lse", "status")}
    n = B.splitkv_paged_workspace_size(desc(), 4) // 4
    f["workspace"] = torch.empty(n + (1 << 16), dtype=torch.int32)
    _apart(lambda a: B.splitkv_paged_decode(desc(), 4, **a, q_stride=512, n_select=3, stream=0), f,
           [("seq_len", (f["o"], 1020)), ("seq_len", (f["lse"], 31)), ("seq_len", (f["workspace"], n - 1)),
            ("page_table", (f["o"], 1023)), ("page_table", (f["lse"], 0)), ("page_table", (f["workspace"], 300)),
            ("pages", (f["o"], 1000)), ("pages", (f["lse"], 30)), ("pages", (f["workspace"], 0)),
            ("lse", (f["pages"], 23)), ("lse", (f["page_table"], 15)), ("lse", (f["seq_len"], 3)),
            ("o", (f["workspace"], 64)), ("lse", (f["workspace"], n - 1)), ("q", (f["workspace"], 128))])


def test_select_writes_apart_from_what_it_reads():
    # Pages 4 x 2 x 3, scratch 4 x 2 x 4 x 2, bounds 10 x 2 x 64 x 2 / 2.
    f = {k: torch.empty(1 << 16, dtype=torch.int32) for k in ("q", "k_bounds", "page_table", "seq_len", "pages", "status", "workspace")}
    _apart(lambda a: B.splitkv_paged_select(desc(), 4, **a, q_stride=512, n_select=3, keep_first=1, keep_last=1, stream=0), f,
           [("pages", (f["workspace"], 63)), ("pages", (f["seq_len"], 3)), ("pages", (f["page_table"], 15)),
            ("pages", (f["q"], 1023)), ("pages", (f["k_bounds"], 1279)), ("seq_len", (f["pages"], 23)),
            ("workspace", (f["pages"], 20)), ("seq_len", (f["workspace"], 60)), ("q", (f["workspace"], 60)),
            ("page_table", (f["workspace"], 63)), ("k_bounds", (f["workspace"], 60))])


def test_append_writes_apart_from_what_it_reads():
    # Five tokens: q_out 5 x 256, k and v 5 x 64, bounds 1280, a rope table of 100 x 64.
    f = {k: torch.empty(1 << 16, dtype=torch.int32)
         for k in ("q", "k", "v", "rope", "page_table", "token_seq", "token_pos", "q_out", "k_cache", "v_cache", "k_bounds", "status")}
    _apart(lambda a: B.splitkv_paged_append(desc(), 4, 5, **a, q_stride=512, k_stride=128, v_stride=128, rope_dim=64, rope_len=100,
                                            interleaved=0, stream=0), f,
           [("rope", (f["q_out"], 1276)), ("page_table", (f["q_out"], 1279)), ("token_seq", (f["q_out"], 1279)),
            ("token_pos", (f["q_out"], 5)), ("k_bounds", (f["q_out"], 1276)), ("q_out", (f["k_bounds"], 1276)),
            ("k", (f["k_bounds"], 1276)), ("v", (f["k_bounds"], 0)), ("q", (f["k_bounds"], 64)), ("rope", (f["k_bounds"], 64)),
            ("token_seq", (f["k_bounds"], 9)), ("token_pos", (f["k_bounds"], 1279)), ("page_table", (f["k_bounds"], 1279)),
            ("k_bounds", (f["rope"], 6396)), ("q_out", (f["token_pos"], 4))])


def test_append_caches_lie_apart():
    f = [torch.empty(1 << 16, dtype=torch.int32) for _ in range(6)]
    with pytest.raises(B.SplitKVError) as e:
        B.splitkv_paged_append(desc(), n_seqs=4, n_tokens=5, q=None, q_stride=0, k=f[0], k_stride=128, v=f[1], v_stride=128,
                               rope=None, rope_dim=0, rope_len=0, interleaved=0, page_table=f[2], token_seq=f[2],
                               token_pos=f[2], q_out=None, k_cache=f[3], v_cache=f[3], k_bounds=None, status=f[4], stream=0)
    assert e.value.code == B.EINVAL


def test_append_refusals():
    f = torch.empty(1 << 16, dtype=torch.int32)
    far = torch.empty(1 << 16, dtype=torch.int32)
    good = dict(n_seqs=4, n_tokens=5, q=f, q_stride=512, k=f, k_stride=128, v=f, v_stride=128, rope=f, rope_dim=64,
                rope_len=100, interleaved=0, page_table=f, token_seq=f, token_pos=f, q_out=far, k_cache=f, v_cache=f,
                k_bounds=f, status=f)
    for kw, code in ((dict(k=None), B.EINVAL), (dict(v=None), B.EINVAL), (dict(q_out=None), B.EINVAL),
                     (dict(page_table=None), B.EINVAL), (dict(token_seq=None), B.EINVAL),
                     (dict(token_pos=None), B.EINVAL), (dict(k_cache=None), B.EINVAL), (dict(v_cache=None), B.EINVAL),
                     (dict(status=None), B.EINVAL), (dict(n_tokens=-1), B.EINVAL), (dict(k_stride=64), B.EINVAL),
                     (dict(v_stride=132), B.EINVAL), (dict(q_stride=256), B.EINVAL), (dict(k=f[1:]), B.EINVAL),
                     (dict(k_bounds=f[1:]), B.EINVAL), (dict(rope=f[1:]), B.EINVAL), (dict(rope_dim=0), B.EINVAL),
                     (dict(rope_dim=63), B.EINVAL), (dict(rope_dim=66), B.EINVAL), (dict(rope_len=0), B.EINVAL),
                     (dict(rope=None), B.EINVAL),                            # rope_dim without a table
                     (dict(q_out=f), B.EINVAL), (dict(q_out=f[128:]), B.EINVAL),  # over q itself
                     (dict(k=far[64:]), B.EINVAL), (dict(v=far[1024:]), B.EINVAL),
                     (dict(n_seqs=-1), B.EINVAL), (dict(n_tokens=1 << 31), B.EUNSUPPORTED)):
        with pytest.raises(B.SplitKVError) as e:
            B.splitkv_paged_append(desc(), **{**good, **kw}, stream=0)
        assert e.value.code == code, kw
    B.splitkv_paged_append(desc(), **{**good, **dict(n_tokens=0, k=None, v=None, q=None, q_out=None)}, stream=0)


def test_select_refusals():
    f = torch.empty(1 << 16, dtype=torch.int32)
    good = dict(n_seqs=4, q=f, q_stride=512, k_bounds=f, page_table=f, seq_len=f, n_select=3, keep_first=1, keep_last=1,
                pages=f, status=f, workspace=f)
    assert B.splitkv_paged_select_workspace_size(desc(), 4) == 4 * 2 * 4 * 8
    assert B.splitkv_paged_select_workspace_size(desc(max_pages=B.PAGED_MAX_SELECT_PAGES + 1), 4) == 0
    for kw, code in ((dict(workspace=None), B.ENOSPACE), (dict(workspace=f[:63]), B.ENOSPACE),
                     (dict(workspace=f[1:]), B.EINVAL), (dict(q=None), B.EINVAL), (dict(k_bounds=None), B.EINVAL), (dict(page_table=None), B.EINVAL),
                     (dict(seq_len=None), B.EINVAL), (dict(pages=None), B.EINVAL), (dict(status=None), B.EINVAL),
                     (dict(n_select=0), B.EINVAL), (dict(keep_first=-1), B.EINVAL), (dict(keep_last=-1), B.EINVAL),
                     (dict(k_bounds=f[2:]), B.EINVAL), (dict(n_select=B.PAGED_MAX_SELECT_PAGES + 1), B.EUNSUPPORTED)):
        with pytest.raises(B.SplitKVError) as e:
            B.splitkv_paged_select(desc(), **{**good, **kw}, stream=0)
        assert e.value.code == code, kw
    with pytest.raises(B.SplitKVError) as e:
        B.splitkv_paged_select(desc(max_pages=B.PAGED_MAX_SELECT_PAGES + 1), **good, stream=0)
    assert e.value.code == B.EUNSUPPORTED
    B.splitkv_paged_select(desc(), **{**good, "n_seqs": 0}, stream=0)


# ------------------------------------------------------------------ the class's refusals
def make(**kw):
    a = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, max_seqs=4, max_pages=6, n_pages=10, bounds=True,
             device="cpu")
    a.update(kw)
    return PagedKV(**a)


def test_class_construction_refusals():
    kv = make()
    assert kv.k_cache.shape == (10, 2, 16, 64) and kv.k_bounds.shape == (10, 2, 2, 64) and kv.dtype == torch.bfloat16
    c = torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16)
    make(n_pages=None, k_cache=c, v_cache=c.clone(), bounds=False)
    t = torch.zeros(10, 16, 2, 64).transpose(1, 2)
    assert make(n_pages=None, k_cache=t, v_cache=torch.zeros(10, 16, 2, 64).transpose(1, 2)).dtype == torch.float32
    for kw in (dict(n_pages=None), dict(n_pages=0), dict(k_cache=c), dict(k_cache=c, v_cache=c[:, :, :8]),
               dict(k_cache=c, v_cache=c.float()), dict(k_cache=c, v_cache=c, n_pages=9),
               dict(k_cache=c, v_cache=c, dtype=torch.float32),
               dict(k_cache=c.expand(10, 2, 16, 64), v_cache=torch.zeros(10, 16, 2, 64, dtype=c.dtype).transpose(1, 2)),
               dict(k_cache=c[..., ::2].repeat(1, 1, 1, 2)[..., :64], v_cache=c, k_bounds=c),
               dict(k_cache=c[:1].expand(10, 2, 16, 64), v_cache=c[:1].expand(10, 2, 16, 64)),  # pages overlap
               dict(dtype=torch.float16), dict(n_q_heads=9), dict(page_size=24), dict(head_dim=130), dict(scale=-1.0),
               dict(max_pages=0), dict(max_seqs=B.PAGED_MAX_SEQS + 1)):
        with pytest.raises(B.SplitKVError):
            make(**kw)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def calls(kv):
    return {
        "decode": (kv.decode, dict(q=bf(3, 8, 64), page_table=i32(3, 6), seq_lens=i32(3))),
        "select": (kv.select, dict(q=bf(3, 8, 64), page_table=i32(3, 6), seq_lens=i32(3), n_select=2)),
        "append": (kv.append, dict(k=bf(5, 2, 64), v=bf(5, 2, 64), page_table=i32(3, 6), token_seq=i32(5), token_pos=i32(5),
                                   q=bf(5, 8, 64), rope=torch.zeros(96, 64))),
    }


@pytest.mark.parametrize("name", ["decode", "select", "append"])
def test_well_formed_calls_reach_the_device_check(name):
    fn, kw = calls(make())[name]
    with pytest.raises(B.SplitKVError, match="not on a CUDA device"):
        fn(**kw)


def _q_strided():
    return bf(3, 16, 64)[:, ::2]


@pytest.mark.parametrize("name,bad", [
    ("decode", dict(q=bf(3, 8, 32))), ("decode", dict(q=bf(2, 8, 64))), ("decode", dict(q=bf(3, 8, 64).float())),
    ("decode", dict(q=bf(3, 64, 8).transpose(1, 2))), ("decode", dict(q=_q_strided())), ("decode", dict(q=bf(3, 512))),
    ("decode", dict(page_table=i32(3, 7))), ("decode", dict(page_table=i32(5, 6))), ("decode", dict(page_table=i32(18))),
    ("decode", dict(page_table=i32(3, 6).long())), ("decode", dict(page_table=i32(6, 3).t())),
    ("decode", dict(page_table=i32(1, 6).expand(3, 6))), ("decode", dict(page_table=i32(3, 0))),
    ("decode", dict(seq_lens=i32(2))), ("decode", dict(seq_lens=i32(3).long())), ("decode", dict(seq_lens=i32(6)[::2])),
    ("decode", dict(pages=i32(3, 2, 0))), ("decode", dict(pages=i32(3, 8, 2))), ("decode", dict(pages=i32(3, 2, 4)[..., :2])),
    ("decode", dict(pages=i32(3, 2, 2).long())), ("decode", dict(o=bf(3, 8, 32))), ("decode", dict(o=bf(8, 3, 64).transpose(0, 1))),
    ("decode", dict(lse=bf(3, 8))), ("decode", dict(lse=torch.zeros(8, 3).t())),
    ("select", dict(n_select=0)), ("select", dict(keep_first=-1)), ("select", dict(keep_last=-2)),
    ("select", dict(pages=i32(3, 2, 3))), ("select", dict(seq_lens=i32(4))), ("select", dict(q=bf(3, 4, 64))),
    ("append", dict(k=bf(5, 8, 64))), ("append", dict(v=bf(4, 2, 64))), ("append", dict(token_seq=i32(4))),
    ("append", dict(token_pos=i32(5).long())), ("append", dict(rope=torch.zeros(96, 64).bfloat16())),
    ("append", dict(rope=torch.zeros(64, 96).t())), ("append", dict(q=None, q_out=bf(5, 8, 64))),
    ("append", dict(q_out=bf(5, 8, 32))), ("append", dict(q=bf(4, 8, 64))), ("append", dict(k=torch.zeros(()).bfloat16())),
])
def test_class_call_refusals(name, bad):
    fn, kw = calls(make())[name]
    with pytest.raises(B.SplitKVError) as e:
        fn(**{**kw, **bad})
    assert e.value.code == B.EINVAL and "CUDA device" not in str(e.value)


def test_select_needs_bounds():
    kv = make(bounds=False)
    with pytest.raises(B.SplitKVError, match="bounds"):
        kv.select(bf(3, 8, 64), i32(3, 6), i32(3), 2)


def test_struct_matches_the_header():
    # The compiler's size of splitkv_paged: four int32, one int64, an int32 (padded), four int64, float, int32.
    assert ctypes.sizeof(B.Paged) == 16 + 8 + 8 + 32 + 8


def test_kernels_launched_early_read_through_coherent_loads():
    # They may be resident while the kernel before them writes what they read: the read-only path is not for that.
    csrc = os.path.join(os.path.dirname(B.__file__), "csrc")
    names = [n for n in os.listdir(csrc) if n.startswith("paged")]
    assert len(names) == 4
    for name in names:
        with open(os.path.join(csrc, name)) as f:
            code = "\n".join(line.split("//")[0] for line in f)
        assert not re.search(r"__ldg|__restrict__|ld\.global\.nc|__constant__", code), name


def test_status_words_are_never_given_back():
    a = make()
    at = a.status.data_ptr()
    assert a.status.shape == (1,) and a.status_value() == 0
    a.status.fill_(3)  # what a graph of its calls may do after it is gone
    others = [make() for _ in range(3)]
    assert len({at, *(x.status.data_ptr() for x in others)}) == 4
    del a
    assert all(x.status_value() == 0 for x in others + [make() for _ in range(300)])


@pytest.mark.parametrize("name", ["k_cache", "v_cache", "k_bounds", "status"])
def test_the_tensors_of_an_object_are_not_replaced(name):
    # The kernels are called with the addresses of those it was made with.
    kv = make()
    held = getattr(kv, name)
    with pytest.raises(AttributeError):
        setattr(kv, name, held.clone())
    assert getattr(kv, name) is held


def test_sizes_past_31_bits_are_not_cut_off():
    kv = make()
    for n in (B.PAGED_MAX_SELECT_PAGES + 1, 1 << 31, (1 << 32) + 2):
        with pytest.raises(B.SplitKVError) as e:
            kv.select(bf(3, 8, 64), i32(3, 6), i32(3), n)
        assert e.value.code == B.EUNSUPPORTED
    for kw in (dict(max_pages=(1 << 32) + 6), dict(n_q_heads=(1 << 32) + 8)):
        with pytest.raises(B.SplitKVError) as e:
            make(**kw)
        assert e.value.code == B.EUNSUPPORTED
    with pytest.raises(B.SplitKVError) as e:
        desc(page_size=(1 << 32) + 16)
    assert e.value.code == B.EUNSUPPORTED


def test_status_words_of_objects_made_in_inference_mode():
    with torch.inference_mode():
        kvs = [make() for _ in range(130)]  # a block of words and more
        kvs[0].status.fill_(1)
    for kv in kvs + [make()]:
        kv.status.zero_()
        assert kv.status_value() == 0
