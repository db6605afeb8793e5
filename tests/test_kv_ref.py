"""The plain form of the 4-bit key/value cache against closed forms, and the host side of the
tq_kv_* calls (sizes, refusals), without a GPU."""
import ctypes as C

import numpy as np
import pytest
import torch

import moe_expert_ffn_q4_amd as tq
from tests import kv_ref


# ---- the plain form ----------------------------------------------------------------------------

@pytest.mark.parametrize("kv,dim,page", [(1, 64, 16), (2, 96, 32), (3, 128, 16), (1, 256, 64)])
def test_layout_is_a_partition(kv, dim, page):
    """Every nibble and every scale of a page belongs to exactly one element (block)."""
    lay = kv_ref.Layout(kv, dim, page)
    nibbles = np.zeros(2 * lay.page_bytes, int)
    for s in range(page):
        for w in (0, 1):
            at, shift, sc = lay.offsets(s, w)
            np.add.at(nibbles, (2 * at + shift // 4).ravel(), 1)
            blocks = sc.reshape(kv, lay.nb, 32)
            assert (blocks == blocks[..., :1]).all()
            for byte in (0, 1):
                for half in (0, 1):
                    np.add.at(nibbles, (2 * (blocks[..., 0] + byte) + half).ravel(), 1)
    assert (nibbles == 1).all()


@pytest.mark.parametrize("kv,dim,page", [(1, 64, 16), (2, 128, 32), (8, 256, 1024)])
def test_page_bytes(kv, dim, page):
    lay = kv_ref.Layout(kv, dim, page)
    d = tq.KvCacheDesc(kv, dim, page, 1, None)
    assert tq.lib().tq_kv_page_bytes(C.byref(d)) == lay.page_bytes == kv * page * dim * 9 // 8


def test_round_block_closed_forms():
    x = np.zeros(32, np.float32)
    assert kv_ref.round_block(x)[0] == 0 and (kv_ref.round_block(x)[1] == 8).all()
    x[5], x[9] = -4.0, 4.0  # the first of the largest stands at -8
    d, n = kv_ref.round_block(x)
    assert d == 0.5 and n[5] == 0 and n[9] == 15 and n[0] == 8
    x[2] = 4.0
    d, n = kv_ref.round_block(x)
    assert d == -0.5 and n[2] == 0 and n[9] == 0 and n[5] == 15
    x = np.full(32, -8.0, np.float32)
    x[1:5] = 0.5, 1.5, -0.5, 2.5  # ties to even
    d, n = kv_ref.round_block(x)
    assert d == 1 and list(n[1:5]) == [8, 10, 8, 10]
    x[7] = np.inf
    assert np.isnan(kv_ref.round_block(x)[0])


def test_write_then_read_is_the_rounding():
    lay = kv_ref.Layout(2, 96, 32)
    g = np.random.default_rng(3)
    data = g.integers(0, 256, 3 * lay.page_bytes, dtype=np.uint8)
    k, v = g.standard_normal((2, 4, 2, 96)).astype(np.float32)
    slots = [95, 0, -1, 33]
    before = data.copy()
    kv_ref.write(data, lay, slots, k, v)
    kr, vr = kv_ref.read(data, lay, slots)
    for x, y in ((k, kr), (v, vr)):
        for r in (0, 1, 3):
            for h in range(2):
                for b in range(3):
                    d, n = kv_ref.round_block(x[r, h, 32 * b:32 * b + 32])
                    assert np.array_equal(y[r, h, 32 * b:32 * b + 32], np.float64(d) * (n - 8))
    touched = np.zeros(data.size, bool)
    for s in (95, 0, 33):
        for w in (0, 1):
            at, _, sc = lay.offsets(s, w)
            for a in (at, sc, sc + 1):
                touched[a.ravel()] = True
    assert np.array_equal(data[~touched], before[~touched])


# ---- refusals ----------------------------------------------------------------------------------

def _cache(kv=2, dim=128, page=16, pages=4, data=4096):
    return tq.KvCacheDesc(kv, dim, page, pages, data)


@pytest.mark.parametrize("kw,code", [
    (dict(kv=0), 2), (dict(kv=1025), 2), (dict(dim=32), 2), (dict(dim=100), 2), (dict(dim=512), 2),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=2048), 2), (dict(pages=0), 2),
    (dict(pages=1 << 27), 2), (dict(data=None), 1), (dict(data=4104), 3),
])
def test_cache_is_checked(kw, code):
    L = tq.lib()
    c = _cache(**kw)
    rows = tq.HeadRows(4096, 2, 256, 128)
    assert L.tq_kv_append(C.byref(c), 0, 1, 4096, C.byref(rows), C.byref(rows), None, None, None, None) == code
    assert L.tq_kv_read(C.byref(c), 0, 1, 4096, 4096, 4096, None) == code
    assert L.tq_last_error()
    if code == 2:
        t = tq.KvStepDesc(1, 1, 0, 16, 32, 48, None, None, 64, 80, None, None, None, None, 96)
        assert L.tq_kv_plan(C.byref(c), C.byref(t), None) == code
    assert L.tq_kv_append(None, 0, 1, 4096, C.byref(rows), C.byref(rows), None, None, None, None) == 1


def test_append_refuses():
    L = tq.lib()
    c = _cache()

    def call(type_=0, rows=1, slots=4096, k=(4096, 2, 256, 128), v=(4096, 2, 256, 128), q=None, qo=None, rope=None):
        r = lambda x: None if x is None else C.byref(tq.HeadRows(*x))  # noqa: E731
        return L.tq_kv_append(C.byref(c), type_, rows, slots, r(k), r(v), r(q), r(qo),
                              None if rope is None else C.byref(rope), None)

    def rope(inv=4096, pos=4096, stride=1, pairs=64, axes=1, sections=(64, 0, 0, 0)):
        return tq.RopeDesc(inv, pos, stride, pairs, axes, (C.c_int64 * 4)(*sections), 0)

    q = (4096, 4, 512, 128)
    assert call(type_=3) == 1 and call(type_=-1) == 1
    assert call(rows=-1) == 2 and call(rows=(1 << 20) + 1) == 2
    assert call(rows=0, slots=None) == 0  # nothing to do
    assert call(slots=None) == 1 and call(slots=4098) == 3
    assert call(k=None) == 1 and call(v=(None, 2, 256, 128)) == 1
    assert call(k=(4096, 3, 256, 128)) == 2 and call(v=(4096, 1, 256, 128)) == 2
    assert call(k=(4098, 2, 256, 128)) == 3 and call(type_=1, k=(4097, 2, 256, 128)) == 3
    assert call(k=(4096, 2, -1, 128)) == 2
    assert call(q=q, qo=q) == 1                       # q without a rope
    assert call(q=q, rope=rope()) == 1                # q without q_out
    assert call(qo=q, rope=rope()) == 1
    assert call(q=q, qo=(8192, 3, 512, 128), rope=rope()) == 2
    assert call(q=(4096, 0, 512, 128), qo=(8192, 0, 512, 128), rope=rope()) == 2
    assert call(rows=2, q=q, qo=(8192, 4, 256, 128), rope=rope()) == 2   # output rows overlap
    assert call(rows=2, q=q, qo=(8192, 4, 512, 64), rope=rope()) == 2    # output heads overlap
    assert call(rows=2, q=q, qo=(4096, 4, 128, 256), rope=rope()) == 1   # in place, other strides
    for bad, code in ((rope(inv=None), 1), (rope(pos=None), 1), (rope(inv=4098), 3), (rope(pairs=0), 2),
                      (rope(pairs=65, sections=(65, 0, 0, 0)), 2), (rope(axes=0), 2), (rope(axes=5), 2),
                      (rope(axes=2, sections=(60, 3, 0, 0)), 2), (rope(axes=2, sections=(65, -1, 0, 0)), 2),
                      (rope(axes=2, stride=-1, sections=(32, 32, 0, 0)), 2)):
        assert call(q=q, qo=q, rope=bad) == code
        assert L.tq_last_error()


def test_read_refuses():
    L = tq.lib()
    c = _cache()
    assert L.tq_kv_read(C.byref(c), 5, 1, 4096, 4096, 4096, None) == 1
    assert L.tq_kv_read(C.byref(c), 0, -1, 4096, 4096, 4096, None) == 2
    assert L.tq_kv_read(C.byref(c), 0, 1, None, 4096, 4096, None) == 1
    assert L.tq_kv_read(C.byref(c), 0, 1, 4096, 4104, 4096, None) == 3
    assert L.tq_kv_read(C.byref(c), 0, 1, 4098, 4096, 4096, None) == 3
    assert L.tq_kv_read(C.byref(c), 0, 0, None, None, None, None) == 0
    assert L.tq_kv_read(C.byref(c), 0, 1, 4096, None, None, None) == 0


def test_plan_refuses():
    L = tq.lib()
    c = _cache(data=None)
    names = [f for f, _ in tq.KvStepDesc._fields_]

    def call(**kw):
        d = dict(requests=3, max_blocks=4, rows=5)
        d.update({f: 4096 + 64 * i for i, f in enumerate(names[3:])})
        d.update(kw)
        return L.tq_kv_plan(C.byref(c), C.byref(tq.KvStepDesc(*[d[f] for f in names])), None)

    for kw in (dict(requests=0), dict(requests=4097), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(rows=-1),
               dict(rows=1 << 28)):
        assert call(**kw) == 2, kw
    for f in names[3:]:
        if f != "free_pages":
            assert call(**{f: None}) == 1, f
        assert call(**{f: 4097}) == 3, f
    for f in names[4:]:
        assert call(**{f: 4096}) == 1, f  # kv_len's memory
    assert L.tq_kv_plan(C.byref(c), None, None) == 1


def _attn(**kw):
    d = dict(rows=1, requests=1, max_blocks=2, q=(4096, 4, 512, 128), out=(8192, 4, 512, 128), lse=None, table=4096,
             seq=4096, cu=4096, scale=0.1, window=0)
    d.update(kw)
    return tq.KvAttnDesc(d["rows"], d["requests"], d["max_blocks"], tq.HeadRows(*d["q"]), tq.HeadRows(*d["out"]),
                         d["lse"], d["table"], d["seq"], d["cu"], d["scale"], d["window"])


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 2), (dict(rows=(1 << 20) + 1), 2), (dict(requests=0), 2), (dict(requests=4097), 2),
    (dict(max_blocks=0), 2), (dict(max_blocks=(1 << 26) + 1), 2), (dict(q=(4096, 3, 512, 128)), 2),
    (dict(q=(4096, 0, 512, 128)), 2), (dict(out=(8192, 2, 512, 128)), 2),
    (dict(q=(4096, 4098, 512, 128), out=(4096, 4098, 512, 128)), 2), (dict(window=-1), 2),
    (dict(window=1 << 31), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=2e30), 1), (dict(q=(None, 4, 512, 128)), 1), (dict(out=(None, 4, 512, 128)), 1),
    (dict(q=(4098, 4, 512, 128)), 3), (dict(table=None), 1), (dict(seq=None), 1), (dict(cu=None), 1),
    (dict(table=4097), 3), (dict(lse=4098), 3), (dict(rows=3, out=(8192, 4, 500, 128)), 2),
    (dict(rows=3, out=(8192, 4, 512, 100)), 2), (dict(q=(4096, 4, -4, 128)), 2),
])
def test_attention_refuses(kw, code):
    L = tq.lib()
    c = _cache()
    assert L.tq_kv_attention(C.byref(c), 0, C.byref(_attn(**kw)), 4096, 1 << 30, None) == code
    assert L.tq_last_error()


def test_attention_workspace_is_checked():
    L = tq.lib()
    c = _cache()
    need = L.tq_kv_attention_workspace_bytes(C.byref(c), 0, C.byref(_attn()))
    assert need > 0
    assert L.tq_kv_attention(C.byref(c), 0, C.byref(_attn()), None, need, None) == 1
    assert L.tq_kv_attention(C.byref(c), 0, C.byref(_attn()), 4096 + 16, need, None) == 3
    assert L.tq_kv_attention(C.byref(c), 0, C.byref(_attn()), 4096, need - 1, None) == 4
    assert L.tq_kv_attention(C.byref(c), 9, C.byref(_attn()), 4096, need, None) == 1
    assert L.tq_kv_attention(C.byref(c), 0, None, 4096, need, None) == 1
    assert L.tq_kv_attention(C.byref(c), 0, C.byref(_attn(rows=0)), None, 0, None) == 0
    assert L.tq_kv_attention_workspace_bytes(C.byref(c), 0, C.byref(_attn(rows=-1))) == 0
    # a long cache and a large batch need no more than a full launch does
    big = L.tq_kv_attention_workspace_bytes(C.byref(c), 0, C.byref(_attn(rows=1000, requests=1000, max_blocks=9999)))
    assert need < big <= 64 << 20


def test_binding_refuses():
    """The binding's own checks, on tensors of the CPU (nothing is launched)."""
    with pytest.raises(ValueError):
        tq.KvCache(2, 100, 16, data=torch.empty((1, 10), dtype=torch.uint8))
    with pytest.raises(ValueError):
        tq.KvCache(2, 128, 16)
    with pytest.raises(ValueError):
        tq.KvCache(2, 128, 16, data=torch.empty((3, 100), dtype=torch.uint8))
    cache = tq.KvCache(2, 128, 16, data=torch.zeros((3, 2 * 16 * 144), dtype=torch.uint8))
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(2, 2, 128)
    with pytest.raises(ValueError, match="int32"):
        tq.kv_append(cache, x, x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="shape"):
        tq.kv_append(cache, x, x[:1], i(0, 1))
    with pytest.raises(ValueError, match="torch.float32"):
        tq.kv_append(cache, x, x.half(), i(0, 1))
    with pytest.raises(ValueError, match="fp32, bf16"):
        tq.kv_append(cache, x.double(), x, i(0, 1))
    with pytest.raises(ValueError, match="dense"):
        tq.kv_append(cache, torch.zeros(2, 2, 256)[..., ::2], x, i(0, 1))
    with pytest.raises(ValueError, match="rope"):
        tq.kv_append(cache, x, x, i(0, 1), q=x)
    with pytest.raises(ValueError, match="not on a GPU"):
        tq.kv_append(cache, x, x, i(0, 1))
    with pytest.raises(ValueError, match="not on a GPU"):
        tq.kv_read(cache, i(0, 1))
    with pytest.raises(ValueError):
        tq.kv_read(cache, i(0, 1), torch.float64)
    with pytest.raises(ValueError, match="together"):
        tq.kv_plan(cache, i(1), i(1), i(1)[None], 1, free_pages=i(0, 1, 2))
    with pytest.raises(ValueError, match="shape"):
        tq.kv_plan(cache, i(1), i(1, 2), i(1)[None], 1)
    with pytest.raises(ValueError, match="multiple"):
        tq.kv_attention(cache, torch.zeros(1, 3, 128), i(0)[None], i(1), i(0, 1))
    with pytest.raises(ValueError, match="shape"):
        tq.kv_attention(cache, x, i(0)[None], i(1), i(0, 1, 2))
    with pytest.raises(ValueError):
        tq.Rope(torch.zeros(4), sections=[1, 2])
    with pytest.raises(ValueError):
        tq.Rope(torch.zeros(4).double())


def test_kernels_use_no_scratch():
    """The compiled kernels of the cache keep everything in registers, at the occupancy that their
    launches count on."""
    import re

    from moe_expert_ffn_q4_amd import build

    least = [(r"k_kv_attnI\w+Li[234]E", 3), (r"k_kv_attnI\w+Li8E", 2), (r"k_kv_wideI\w+Li[234]E", 2),
             (r"k_kv_wideI\w+Li8E", 1), (r"k_kv_(plan|append|read|join)", 4)]
    resources = build.kernel_resources()
    for pattern, occupancy in least:
        hits = {k: v for k, v in resources.items() if re.search(pattern, k)}
        assert hits, pattern
        for name, r in hits.items():
            assert r["scratch"] == 0, f"{name}: {r['scratch']} bytes of scratch per lane"
            assert r["occupancy"] >= occupancy, f"{name}: occupancy {r['occupancy']} < {occupancy}"
