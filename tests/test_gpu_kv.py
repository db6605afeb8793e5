"""GPU parity of the paged 4-bit key/value cache (plan, append, read, attention) with its plain
form in 64 bits (tests/kv_ref.py).

Append and plan are held bitwise (the rounding is defined exactly; keys are turned in fp64 on both
sides, so their fp32 roundings agree but for a 2^-29 chance a value). Attention is held to
kv_ref.attention's bound plus the weights' rounding (half a step of fp16: 2^-11 of the weights'
sum of magnitudes for bf16 activations, whose weights are one fp16 term; 2^-21 for the two terms of
fp32 and fp16) and half a step of the output type."""
import numpy as np
import pytest
import torch

from tests import kv_ref
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("moe_expert_ffn_q4_amd")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WEIGHT = {"f32": 2.0**-21, "bf16": 2.0**-11, "f16": 2.0**-21}
I32 = dict(dtype=torch.int32, device="cuda:0")


def _case(*a):
    print("case:", *a, flush=True)


def i32(v):
    return torch.tensor(np.asarray(v), **I32)


def rounded(x, t):
    """fp64 array -> (tensor of type t on the GPU, its values in fp64)."""
    y = torch.from_numpy(np.asarray(x, np.float64)).to(TYPES[t])
    return y.to("cuda:0"), y.double().numpy()


def filled_cache(g, lay, pages, scale=0.3, junk=0xFF):
    """(flat uint8 array, KvCache): every byte `junk` (0xFF: scales that are not numbers)."""
    data = np.full(pages * lay.page_bytes, junk, np.uint8)
    return data


def put(g, data, lay, slots, scale=0.3, spread=1.0):
    """Random blocks into slots: nibbles uniform, scales +-scale * spread^u."""
    for s in slots:
        for w in (0, 1):
            at, shift, sc = lay.offsets(int(s), w)
            n = g.integers(0, 16, at.shape)
            lo = shift == 0
            np.bitwise_and.at(data, at.ravel(), np.where(lo, 0xF0, 0x0F).ravel().astype(np.uint8))
            np.bitwise_or.at(data, at.ravel(), (n << shift).ravel().astype(np.uint8))
            d = scale * spread ** g.uniform(-1, 1, (lay.kv, lay.nb)) * g.choice([-1, 1], (lay.kv, lay.nb))
            bits = d.astype(np.float16).view(np.uint16)
            first = sc.reshape(lay.kv, lay.nb, 32)[..., 0]
            data[first], data[first + 1] = bits & 255, bits >> 8


def cache_of(data, lay, page):
    return tq.KvCache(lay.kv, lay.dim, page, data=dev(data.reshape(-1, lay.page_bytes)))


class Batch:
    """Requests of given lengths in scattered pages, with junk everywhere else."""

    def __init__(self, g, kv, dim, page, lens, scale=0.3, spread=1.0, extra=2):
        self.lay, self.page, self.lens = kv_ref.Layout(kv, dim, page), page, list(lens)
        have = [-(-n // page) for n in lens]
        self.pages = sum(have) + extra
        order = g.permutation(self.pages)
        mb = max(have + [1]) + 1
        self.table = np.full((len(lens), mb), -1)
        at = 0
        for r, n in enumerate(have):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.data = filled_cache(g, self.lay, self.pages)
        for r in range(len(lens)):
            put(g, self.data, self.lay, self.slots(r), scale, spread)

    def slots(self, r):
        t = np.arange(self.lens[r])
        return self.table[r, t // self.page] * self.page + t % self.page

    def rows(self, r):
        return kv_ref.read(self.data, self.lay, self.slots(r))


def check_attention(b, q64, got, lse, news, t, scale, window, hidden=None):
    cu = np.concatenate([[0], np.cumsum(news)])
    kv = [b.rows(r) for r in range(len(b.lens))]
    ref, rlse, tol, ltol, mag = kv_ref.attention(q64, lambda r: kv[r][0], lambda r: kv[r][1], b.lens, cu, b.lay.kv,
                                                 scale, window, hidden)
    n = cu[-1]
    tol = tol + 2 * WEIGHT[t] * mag + torch.finfo(TYPES[t]).eps / 2 * np.abs(ref) + 1e-30
    if t == "f16":
        tol = tol + 2.0**-25  # half a step of the smallest fp16
    got, lse = got.astype(np.float64)[:n], lse.astype(np.float64)[:n]
    ref, rlse, tol, ltol = ref[:n], rlse[:n], tol[:n], ltol[:n]
    assert np.array_equal(np.isneginf(lse), np.isneginf(rlse))
    fin = np.isfinite(rlse)
    assert (np.abs(lse[fin] - rlse[fin]) <= ltol[fin]).all(), f"lse off by {np.max(np.abs(lse[fin] - rlse[fin]) / ltol[fin])}"
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {np.max(err / tol)} of the bound at {np.unravel_index(np.argmax(err / tol), err.shape)}"
    return float(np.max(err / tol)) if err.size else 0.0


def run_attention(b, q, news, scale=None, window=0, **kw):
    cu = np.concatenate([[0], np.cumsum(news)])
    cache = cache_of(b.data, b.lay, b.page)
    out, lse = tq.kv_attention(cache, q, i32(b.table), i32(b.lens), i32(cu), scale=scale, window=window,
                               return_lse=True, **kw)
    return host(out.double()), host(lse)


def attention_case(seed, t, kv, G, dim, page, lens, news, window=0, qscale=1.5, scale=0.3, spread=1.0):
    g = np.random.default_rng(seed)
    b = Batch(g, kv, dim, page, lens, scale, spread)
    q, q64 = rounded(qscale * g.standard_normal((sum(news), kv * G, dim)), t)
    out, lse = run_attention(b, q, news, window=window)
    return check_attention(b, q64, out, lse, news, t, dim**-0.5, window)


# ---- read and append -----------------------------------------------------------------------------

@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kv,dim,page", [(1, 64, 16), (3, 96, 32), (2, 128, 64), (2, 256, 16)])
def test_read(kv, dim, page, t):
    _case("read", kv, dim, page, t)
    g = np.random.default_rng(dim + kv)
    lay = kv_ref.Layout(kv, dim, page)
    data = filled_cache(g, lay, 3)
    put(g, data, lay, range(3 * page))
    slots = np.concatenate([g.permutation(3 * page)[:37], [-1, 3 * page, 5, 5, 2**31 - 1, -2**31]])
    k, v = tq.kv_read(cache_of(data, lay, page), i32(slots), TYPES[t])
    kr, vr = kv_ref.read(data, lay, slots)
    for got, ref in ((k, kr), (v, vr)):
        assert torch.equal(got.cpu(), torch.from_numpy(ref).to(TYPES[t]))


def append_case(seed, t, rows, kv, heads, dim, page, sections, pairs, interleaved, strided=False, special=None,
                in_place=False):
    g = np.random.default_rng(seed)
    lay = kv_ref.Layout(kv, dim, page)
    pages = -(-rows // page) + 2
    data = g.integers(0, 256, pages * lay.page_bytes, dtype=np.uint8)
    slots = g.permutation(pages * page)[:rows]
    if rows > 3:
        slots[1], slots[rows // 2] = -1, pages * page  # not written
    total = heads + 2 * kv
    x = g.standard_normal((rows, total, dim))
    if special is not None:
        special(x, heads, kv, g)
    with np.errstate(over="ignore"):
        xt, x64 = rounded(x, t)
    if strided:  # heads first, rows inside, at an odd offset
        buf = torch.zeros((total, rows, dim + 1), dtype=TYPES[t], device="cuda:0")
        buf[..., 1:] = xt.transpose(0, 1)
        xt = buf[..., 1:].transpose(0, 1)
    q, k, v = xt.split([heads, kv, kv], dim=1)
    positions = g.integers(0, 1 << 20, (len(sections), rows))
    inv = (10000.0 ** (-np.arange(pairs) / max(1, pairs))).astype(np.float32)
    cache = cache_of(data, lay, page)
    live = (slots >= 0) & (slots < pages * page)
    if pairs:
        rope = tq.Rope(dev(inv), sections, interleaved)
        out = q if in_place else torch.full(q.shape, 7.0, dtype=TYPES[t], device="cuda:0")
        before = out.clone()
        tq.kv_append(cache, k, v, i32(slots), q=q, rope=rope, positions=i32(positions), q_out=out)
        turned = kv_ref.turn(x64[:, :heads + kv], positions, inv, sections, interleaved)
        want = torch.from_numpy(turned[:, :heads])
        got = out.cpu()
        assert torch.equal(got[~live], before.cpu()[~live])
        # half a step of the type (and of its smallest numbers) behind fp32 arithmetic: cosine and sine
        # to 2^-24 of at most 1 each, two products and their sum to 2^-24 each of at most |a| + |b|
        q64 = torch.from_numpy(x64[:, :heads])
        part = q64.abs().amax(-1, keepdim=True) * 2
        tol = torch.finfo(TYPES[t]).eps / 2 * want.abs() * (1 + 2.0**-20) + {"f32": 2.0**-149, "bf16": 2.0**-133, "f16": 2.0**-25}[t]
        tol = tol + 4 * 2.0**-24 * part
        diff = (got.double() - want).abs()
        assert bool((diff <= tol)[live].all())
        k32 = turned[:, heads:].astype(np.float32)
    else:
        assert tq.kv_append(cache, k, v, i32(slots)) is None
        k32 = x64[:, heads:heads + kv].astype(np.float32)
    ref = data.copy()
    kv_ref.write(ref, lay, slots, k32, x64[:, heads + kv:].astype(np.float32))
    got = host(cache.data).ravel()
    # scales that are not numbers compare as such
    bad = np.nonzero(got != ref)[0]
    assert bad.size == 0, f"{bad.size} bytes differ, first at {bad[:4]}: {got[bad[:4]]} for {ref[bad[:4]]}"


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,kv,heads,dim,page,sections,pairs,interleaved", [
    (1, 2, 8, 128, 16, [64], 64, False),
    (5, 1, 3, 64, 16, [32], 32, True),
    (33, 2, 4, 96, 32, [20, 12, 16], 48, False),      # three axes
    (17, 3, 3, 128, 64, [8, 8, 8, 8], 32, True),       # part of the head, four axes
    (7, 2, 2, 256, 16, [0, 100], 100, False),          # an empty axis, pairs 100 of 128
    (9, 1, 2, 64, 16, [7], 7, False),                  # an odd number of pairs: one at a time
    (600, 2, 4, 64, 16, [32], 32, False),              # several rows per workgroup
    (70, 20, 40, 64, 32, [32], 32, True),              # more heads than a workgroup takes
    (40, 2, 0, 128, 16, [0], 0, False),                # no rope
])
def test_append(rows, kv, heads, dim, page, sections, pairs, interleaved, t):
    _case("append", rows, kv, heads, dim, page, sections, pairs, interleaved, t)
    if heads == 0:
        heads = 1 if pairs else 0
    append_case(rows, t, rows, kv, heads, dim, page, sections, pairs, interleaved)


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_strided_rows(t, in_place):
    _case("append strided", t, in_place)
    append_case(5, t, 21, 2, 6, 128, 16, [64], 64, False, strided=True, in_place=in_place)
    append_case(6, t, 21, 2, 6, 128, 16, [64], 64, True, strided=False, in_place=in_place)


@pytest.mark.parametrize("kind", ["ties", "zeros", "tiny", "huge", "odd"])
def test_append_special_values(kind):
    """Blocks whose rounding has ties, zeros, scales below fp16's normal range or above its
    largest, and values that are not finite (the block then reads as not numbers)."""
    _case("append special", kind)

    def special(x, heads, kv, g):
        v = x[:, heads:]
        if kind == "ties":  # largest magnitudes of both signs, and quotients half-way
            v[:] = g.integers(-16, 17, v.shape) * 0.25
        elif kind == "zeros":
            v[::2] = 0.0
            v[1::2] *= 1e-9
        elif kind == "tiny":
            v *= 10.0 ** g.uniform(-9, -4, v.shape[:2] + (1,))
        elif kind == "huge":
            v *= 10.0 ** g.uniform(4, 38, v.shape[:2] + (1,))
        else:
            v[::3, 0, 5], v[1::3, 1, 40], v[2::5, 0, 64] = np.nan, np.inf, -np.inf

    append_case(11, "f32", 40, 2, 0, 128, 16, [0], 0, False, special=special)


def test_append_nothing():
    cache = tq.KvCache(2, 64, 16, pages=2)
    cache.data.fill_(3)
    x = torch.zeros((0, 2, 64), device="cuda:0")
    assert tq.kv_append(cache, x, x, i32(np.zeros(0))) is None
    x = torch.randn((4, 2, 64), device="cuda:0")
    tq.kv_append(cache, x, x, i32([-1, 32, 1 << 30, -7]))
    assert bool((cache.data == 3).all())
    k, v = tq.kv_read(cache, i32(np.zeros(0)))
    assert k.shape == (0, 2, 64)


def test_slots_past_32_bits():
    """A cache of more than 4 GiB: rows near its end are written, read and attended where they
    belong."""
    _case("past 32 bits")
    g = np.random.default_rng(8)
    lay = kv_ref.Layout(8, 256, 64)
    pages = (5 << 30) // lay.page_bytes
    cache = tq.KvCache(8, 256, 64, pages=pages)
    far = np.array([pages - 1, pages - 3, 1])
    t = np.arange(150)
    slots = far[t // 64] * 64 + t % 64
    k, v = g.standard_normal((2, 150, 8, 256)).astype(np.float32)
    tq.kv_append(cache, dev(k), dev(v), i32(slots))
    small = np.zeros(3 * lay.page_bytes, np.uint8)
    kv_ref.write(small, lay, t, k, v)
    kr, vr = kv_ref.read(small, lay, t)
    kg, vg = tq.kv_read(cache, i32(slots))
    assert np.array_equal(host(kg), kr.astype(np.float32)) and np.array_equal(host(vg), vr.astype(np.float32))
    q, q64 = rounded(g.standard_normal((1, 8, 256)), "f32")
    out, lse = tq.kv_attention(cache, q, i32(far[None]), i32([150]), i32([0, 1]), return_lse=True)
    b = Batch.__new__(Batch)
    b.lay, b.lens, b.rows = lay, [150], lambda r: (kr, vr)
    check_attention(b, q64, host(out.double()), host(lse), [1], "f32", 256**-0.5, 0)


# ---- plan ------------------------------------------------------------------------------------------

def plan_case(kv, new, page, rows, mb=None, pages=None, managed=True, count=None, table=None, seed=0):
    g = np.random.default_rng(seed)
    kv, new = np.asarray(kv), np.asarray(new)
    have = -(-np.maximum(kv, 0) // page)
    after = -(-(np.maximum(kv, 0) + np.maximum(new, 0)) // page)
    mb = mb or int(max(after.max(), have.max(), 1)) + 1
    used = int(have.sum() if managed else after.sum())
    pages = pages or used + int((after - have).sum()) + 3
    order = g.permutation(max(pages, used))
    if table is None:
        table = np.full((len(kv), mb), -1)
        at = 0
        for r in range(len(kv)):
            n = min(int(have[r] if managed else after[r]), mb)
            table[r, :n] = order[at:at + n]
            at += n
    free = np.full(pages, -9)
    rest = order[used:][:pages]
    free[:len(rest)] = rest
    count = len(rest) if count is None else count
    cache = tq.KvCache(1, 64, page, pages=pages)
    td, fd = i32(table), i32(free)
    ref = kv_ref.plan(kv, new, table, rows, page, pages, free if managed else None, count if managed else None)
    for again in range(2):  # a repeated call gives the same
        got = tq.kv_plan(cache, i32(kv), i32(new), td, rows, fd if managed else None, i32([count]) if managed else None)
        assert set(got) == set(ref)
        for f in ref:
            assert np.array_equal(host(got[f]), ref[f]), (f, again, host(got[f]), ref[f])
    return ref


@pytest.mark.parametrize("kv,new,page,rows", [
    ([0], [1], 16, 1),
    ([15], [1], 16, 3),
    ([16], [1], 16, 1),
    ([0, 5, 64, 63], [130, 0, 1, 2], 64, 140),
    ([100, 7, 33, 0, 64], [-1, 1, -1, 40, 1], 32, 42),     # ended requests' pages go to the others
    ([10, 0], [-1, 0], 16, 0),                              # nothing new
    ([0, 0, 0], [0, 0, 0], 16, 4),
    ([1000], [1], 1024, 1),
])
@pytest.mark.parametrize("managed", [True, False])
def test_plan(kv, new, page, rows, managed):
    _case("plan", kv, new, page, rows, managed)
    assert plan_case(kv, new, page, rows, managed=managed)["status"][0] == 0


@pytest.mark.parametrize("n,page", [(255, 16), (256, 32), (257, 16), (1000, 64), (4096, 16)])
def test_plan_many(n, page):
    _case("plan many", n, page)
    g = np.random.default_rng(n)
    kv = g.integers(0, 300, n)
    new = np.where(g.random(n) < 0.1, -1, np.where(g.random(n) < 0.1, g.integers(0, 90, n), 1))
    rows = int(np.maximum(new, 0).sum()) + 11
    for managed in (True, False):
        assert plan_case(kv, new, page, rows, managed=managed, seed=n)["status"][0] == 0


@pytest.mark.parametrize("kw,status", [
    (dict(kv=[5, 5], new=[60, 1], count=2), 1),
    (dict(kv=[5, 5], new=[60, 1], rows=60), 2),
    (dict(kv=[5, 5], new=[60, 1], mb=3), 4),
    (dict(kv=[50, 5], new=[-1, 1], mb=3), 4),
    (dict(kv=[-1, 5], new=[60, 1]), 8),
    (dict(kv=[5, 5], new=[-2, 1]), 8),
    (dict(kv=[5, 5], new=[1, 1], count=-1), 8),
    (dict(kv=[5, 5], new=[1, 1], count=10**6), 8),
    (dict(kv=[40, 5], new=[-1, 1], pages=6, count=5), 8),   # more pages come back than there are
    (dict(kv=[2**31 - 1, 5], new=[2**31 - 1, 1], mb=3, pages=9, count=0), 4 | 2 | 1),
])
def test_plan_says_why_nothing_was_done(kw, status):
    _case("plan status", kw)
    kw = dict(kw)
    args = dict(page=16, rows=kw.pop("rows", 80))
    if kw["kv"][0] > 2**30:
        kw["table"] = np.zeros((2, 3), int)
        g = kw.pop("pages")
        cache = tq.KvCache(1, 64, 16, pages=g)
        table, free = i32(kw["table"]), i32(np.arange(g))
        got = tq.kv_plan(cache, i32(kw["kv"]), i32(kw["new"]), table, 80, free, i32([0]))
        assert int(got["status"]) == status
        assert bool((got["slots"] == -1).all()) and np.array_equal(host(got["seq_len"]), kw["kv"])
        return
    assert plan_case(**args, **kw)["status"][0] == status


def test_plan_marks_bad_pages():
    """Page numbers outside the cache (in a table or on the stack) give slot -1."""
    table = np.array([[0, 99, 2], [-5, 1, 1]])
    ref = plan_case([20, 3], [14, 2], 16, 16, table=table, pages=4, managed=False)
    assert (ref["slots"][:12] == -1).all() and (ref["slots"][14:] == -1).all()


# ---- attention ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kv,G,dim,page", [(1, 1, 64, 16), (2, 4, 128, 64), (1, 8, 128, 16), (2, 3, 96, 32),
                                           (1, 16, 64, 32), (1, 5, 256, 16), (1, 20, 128, 64), (3, 7, 64, 128)])
def test_attention_one_token(kv, G, dim, page, t):
    _case("attention decode", kv, G, dim, page, t)
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 257, 1001]
    r = attention_case(dim + G, t, kv, G, dim, page, lens, [1] * len(lens))
    print("worst of the bound:", r)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("window", [0, 1, 16, 50])
@pytest.mark.parametrize("kv,G,dim", [(2, 4, 64), (1, 3, 128), (1, 12, 96)])
def test_attention_several_tokens(kv, G, dim, window, t):
    _case("attention several", kv, G, dim, window, t)
    lens = [3, 40, 129, 200, 77, 64]
    news = [3, 5, 1, 70, 0, 64]
    attention_case(window + G, t, kv, G, dim, 16, lens, news, window)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_attention_long(t):
    """A sequence cut over many workgroups, beside short ones."""
    _case("attention long", t)
    attention_case(1, t, 2, 4, 128, 64, [9000, 3, 500], [1, 1, 2])
    attention_case(2, t, 1, 2, 64, 16, [20011], [1], qscale=4.0)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale,spread,qscale", [(6000.0, 1.3, 1e-4), (1e-5, 8.0, 1e5), (0.1, 300.0, 0.3),
                                                 (0.3, 1.0, 12.0), (0.3, 1.0, 0.0)])
def test_attention_ranges(scale, spread, qscale, t):
    """Scales over fp16's whole range in one row, peaked and flat softmax, zero queries."""
    _case("attention ranges", scale, spread, qscale, t)
    if t == "f16" and qscale == 1e5:
        qscale = 1e4
    attention_case(7, t, 2, 4, 64, 16, [700, 90], [1, 3], qscale=qscale, scale=scale, spread=spread)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_attention_rows_without_tokens(t):
    """Requests of length zero, requests without new tokens, more new tokens than the sequence has
    (the first see nothing), and rows behind the last request."""
    _case("attention empty rows", t)
    g = np.random.default_rng(4)
    b = Batch(g, 2, 64, 16, [0, 40, 2, 0, 7])
    news = [1, 0, 4, 0, 2]
    q, q64 = rounded(g.standard_normal((sum(news) + 3, 4, 64)), t)
    out = torch.full(q.shape, 5.0, dtype=TYPES[t], device="cuda:0")
    got, lse = run_attention(b, q, news, out=out)
    assert (got[0] == 0).all() and np.isneginf(lse[0]).all()
    assert (got[1:3] == 0).all() and np.isneginf(lse[1:3]).all()
    assert (got[7:] == 5).all()
    check_attention(b, q64, got, lse, news, t, 64**-0.5, 0)


def test_attention_values_that_are_not_numbers():
    """A key or value that is not a number reaches the rows that see it and no other."""
    _case("attention nan")
    g = np.random.default_rng(5)
    for which in (0, 1):
        b = Batch(g, 1, 64, 16, [50, 60])
        news = [8, 1]
        slot = b.slots(0)[46]  # seen by the rows of tokens 46..49 only
        _, _, sc = b.lay.offsets(int(slot), which)
        b.data[sc[0, 0]], b.data[sc[0, 0] + 1] = 0x00, 0x7E
        for t in TYPES:
            q, q64 = rounded(g.standard_normal((9, 2, 64)), t)
            out, lse = run_attention(b, q, news)
            assert np.isnan(out[4:8, :, :32]).all()
            assert np.isfinite(out[:4]).all() and np.isfinite(out[8:]).all() and np.isfinite(lse[:4]).all()
            good = Batch.__new__(Batch)
            good.lay, good.lens = b.lay, [46, 60]
            good.rows = lambda r, b=b: tuple(x[:good.lens[r]] for x in b.rows(r))
            keep = [0, 1, 2, 3, 8]
            check_attention(good, q64[keep], out[keep], lse[keep], [4, 1], t, 64**-0.5, 0)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kv,G,dim,page,lens,news,window", [
    (1, 4, 128, 16, [200], [200], 0),                    # a prompt from nothing
    (2, 1, 64, 32, [300, 33, 170], [130, 33, 170], 0),   # one head a group: 130 columns are two tiles
    (1, 5, 96, 64, [260, 1], [77, 1], 40),               # a window; tiles of 125 of 128 columns
    (1, 3, 256, 16, [150, 90], [150, 30], 0),
    (1, 160, 64, 16, [70], [3], 0),                      # more heads than a tile has columns
    (2, 8, 128, 64, [3000, 60], [40, 60], 0),            # cut over workgroups
])
def test_attention_prompts(kv, G, dim, page, lens, news, window, t):
    """Requests with many new tokens, whose tiles share unpacked keys and values."""
    _case("attention prompts", kv, G, dim, page, lens, news, window, t)
    attention_case(dim + window, t, kv, G, dim, page, lens, news, window)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale,spread,qscale", [(6000.0, 1.3, 1e-4), (1e-5, 8.0, 1e4), (0.1, 300.0, 0.3),
                                                 (0.3, 1.0, 12.0), (0.3, 1.0, 0.0)])
def test_attention_prompt_ranges(scale, spread, qscale, t):
    _case("attention prompt ranges", scale, spread, qscale, t)
    attention_case(17, t, 2, 4, 64, 16, [250, 90], [50, 33], qscale=qscale, scale=scale, spread=spread)


def test_attention_prompt_values_that_are_not_numbers():
    """Keys and values that are not numbers, and junk behind the last token, in a prompt's tiles: they
    reach the rows that see them, a value only in its block's dimensions."""
    _case("attention prompt nan")
    g = np.random.default_rng(15)
    for which in (0, 1):
        b = Batch(g, 1, 64, 16, [120, 75])
        news = [100, 75]
        slot = b.slots(0)[46]  # seen by the tokens from 46 on: rows 26 .. 99 of the request
        _, _, sc = b.lay.offsets(int(slot), which)
        b.data[sc[0, 32]], b.data[sc[0, 32] + 1] = 0x00, 0x7E
        good = Batch.__new__(Batch)
        good.lay, good.lens = b.lay, [46, 75]
        good.rows = lambda r, b=b: tuple(x[:good.lens[r]] for x in b.rows(r))
        for t in TYPES:
            q, q64 = rounded(g.standard_normal((175, 2, 64)), t)
            out, lse = run_attention(b, q, news)
            hit = out[26:100, :, 32:] if which else out[26:100]
            assert np.isnan(hit).all()
            if which:
                assert np.isfinite(out[26:100, :, :32]).all() and np.isfinite(lse).all()
            keep = list(range(26)) + list(range(100, 175))
            check_attention(good, q64[keep], out[keep], lse[keep], [26, 75], t, 64**-0.5, 0)


def test_attention_prompt_pages_outside_the_cache():
    _case("attention prompt bad pages")
    g = np.random.default_rng(16)
    b = Batch(g, 2, 128, 16, [100, 64])
    rows = [b.rows(r) for r in range(2)]
    hidden = [np.zeros(n, bool) for n in b.lens]
    for r, col, page in ((0, 1, -1), (0, 4, b.pages), (0, 5, 10**6), (1, 0, 2**31 - 1)):
        b.table[r, col] = page
        hidden[r][16 * col:16 * col + 16] = True
    b.rows = lambda r: rows[r]
    news = [60, 64]
    for t in TYPES:
        q, q64 = rounded(g.standard_normal((124, 4, 128)), t)
        out, lse = run_attention(b, q, news)
        check_attention(b, q64, out, lse, news, t, 128**-0.5, 0, hidden=lambda r: hidden[r])


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_attention_prompt_rows_behind(t):
    """Prompts beside single tokens and requests without tokens; rows behind the last one and an output
    with strides are left alone; the same call gives the same bits."""
    _case("attention prompt rows", t)
    g = np.random.default_rng(18)
    b = Batch(g, 2, 64, 32, [0, 140, 55, 2, 64])
    news = [0, 90, 1, 4, 64]
    q, q64 = rounded(g.standard_normal((sum(news) + 5, 8, 64)), t)
    outs = []
    for _ in range(3):
        wide = torch.full((sum(news) + 5, 10, 64), 5.0, dtype=TYPES[t], device="cuda:0")
        got, lse = run_attention(b, q, news, out=wide[:, 1:9])
        assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 9] == 5).all()) and (got[sum(news):] == 5).all()
        outs.append(wide)
    assert all(torch.equal(outs[0], o) for o in outs)
    check_attention(b, q64, got, lse, news, t, 64**-0.5, 0)


def test_attention_query_that_is_not_a_number():
    _case("attention nan query")
    g = np.random.default_rng(6)
    for t in TYPES:
        b = Batch(g, 1, 128, 16, [77])
        x = g.standard_normal((3, 4, 128))
        x[1, 2, 7] = np.nan
        x[2, 0, 7] = np.inf
        q, _ = rounded(x, t)
        x2 = x.copy()
        x2[1, 2] = x2[2, 0] = 0
        q2, _ = rounded(x2, t)
        out, _ = run_attention(b, q, [3])
        clean, _ = run_attention(b, q2, [3])
        bad = np.zeros((3, 4), bool)
        bad[1, 2] = bad[2, 0] = True
        assert np.isnan(out[bad]).all() and np.array_equal(out[~bad], clean[~bad])


def test_attention_prompt_query_that_is_not_a_number():
    _case("attention prompt nan query")
    g = np.random.default_rng(19)
    b = Batch(g, 1, 64, 16, [90])
    for t in TYPES:
        x = g.standard_normal((50, 4, 64))
        bad = np.zeros((50, 4), bool)
        bad[3, 1] = bad[47, 2] = True
        x2 = x.copy()
        x[3, 1, 7], x[47, 2, 60] = np.nan, np.inf
        x2[bad] = 0
        out, _ = run_attention(b, rounded(x, t)[0], [50])
        clean, _ = run_attention(b, rounded(x2, t)[0], [50])
        assert np.isnan(out[bad]).all() and np.array_equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_attention_tiny_scale(t):
    """A scale and queries so small that every logit is 0, beside hidden tokens: plain means."""
    _case("attention tiny scale", t)
    g = np.random.default_rng(20)
    b = Batch(g, 1, 64, 16, [45, 60])
    for news in ([2, 1], [45, 40]):
        q, q64 = rounded(1e-7 * g.standard_normal((sum(news), 4, 64)), t)
        if t != "f16":
            q, q64 = rounded(1e-30 * g.standard_normal((sum(news), 4, 64)), t)
        out, lse = run_attention(b, q, news, scale=1e-25)
        check_attention(b, q64, out, lse, news, t, 1e-25, 0)


def test_attention_a_window_past_every_token():
    """The largest window there is, with more new tokens than the sequence has."""
    _case("attention large window")
    g = np.random.default_rng(21)
    b = Batch(g, 1, 64, 16, [3, 50])
    for t in TYPES:
        q, q64 = rounded(g.standard_normal((52, 2, 64)), t)
        out, lse = run_attention(b, q, [5, 47], window=2**31 - 1)
        check_attention(b, q64, out, lse, [5, 47], t, 64**-0.5, 0)


def test_attention_pages_outside_the_cache():
    """Their tokens count as masked; nothing outside the cache is read."""
    _case("attention bad pages")
    g = np.random.default_rng(9)
    b = Batch(g, 2, 128, 16, [100, 64, 30])
    rows = [b.rows(r) for r in range(3)]
    hidden = [np.zeros(n, bool) for n in b.lens]
    for r, col, page in ((0, 1, -1), (0, 4, b.pages), (1, 0, 2**31 - 1), (2, 0, -2**31), (2, 1, 10**6)):
        b.table[r, col] = page
        hidden[r][16 * col:16 * col + 16] = True
    b.rows = lambda r: rows[r]
    news = [2, 1, 1]
    for t in TYPES:
        q, q64 = rounded(g.standard_normal((4, 4, 128)), t)
        out, lse = run_attention(b, q, news)
        check_attention(b, q64, out, lse, news, t, 128**-0.5, 0, hidden=lambda r: hidden[r])
        assert (out[3] == 0).all()


def test_attention_strides_and_scale():
    """Queries inside a wider buffer, heads before rows, an output with strides, another scale."""
    _case("attention strides")
    g = np.random.default_rng(10)
    for t in TYPES:
        b = Batch(g, 2, 64, 32, [70, 33])
        news = [2, 3]
        _, q64 = rounded(g.standard_normal((5, 6, 64)), t)
        wide = torch.zeros((6, 5, 65), dtype=TYPES[t], device="cuda:0")
        wide[..., 1:] = torch.from_numpy(q64).to(TYPES[t]).transpose(0, 1).to("cuda:0")
        q = wide[..., 1:].transpose(0, 1)
        o = torch.full((5, 9, 64), 3.0, dtype=TYPES[t], device="cuda:0")
        out, lse = run_attention(b, q, news, scale=0.31, out=o[:, 2:8])
        check_attention(b, q64, out, lse, news, t, 0.31, 0)
        assert bool((o[:, :2] == 3).all()) and bool((o[:, 8:] == 3).all())


def test_attention_repeats_bitwise():
    _case("attention repeats")
    g = np.random.default_rng(12)
    b = Batch(g, 2, 128, 64, [5000, 17, 900])
    q, _ = rounded(g.standard_normal((3, 8, 128)), "f32")
    first = run_attention(b, q, [1, 1, 1])
    for _ in range(20):
        again = run_attention(b, q, [1, 1, 1])
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_attention_on_two_streams():
    """Calls on two streams at once, each with the workspace of its own stream."""
    _case("attention streams")
    g = np.random.default_rng(13)
    b = [Batch(g, 2, 128, 64, [3000 + 100 * i, 40]) for i in range(2)]
    q = [rounded(g.standard_normal((2, 8, 128)), "bf16")[0] for _ in range(2)]
    want = [run_attention(b[i], q[i], [1, 1]) for i in range(2)]
    caches = [cache_of(x.data, x.lay, x.page) for x in b]
    args = [(i32(x.table), i32(x.lens), i32([0, 1, 2])) for x in b]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i in range(2):
            got[i].append(tq.kv_attention(caches[i], q[i], *args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert np.array_equal(host(o.double()), want[i][0])


@pytest.mark.parametrize("bad", [{"scale": -1.0}, {"window": -1}])
def test_attention_after_a_refused_call(bad):
    """A refused call leaves nothing behind: the next one of the same sizes runs."""
    _case(f"attention refused {bad}")
    g = np.random.default_rng(14)
    b = Batch(g, 2, 64, 16, [40, 3])
    q, q64 = rounded(g.standard_normal((2, 4, 64)), "f32")
    cache = cache_of(b.data, b.lay, b.page)
    args = (q, i32(b.table), i32(b.lens), i32([0, 1, 2]))
    with pytest.raises(tq.TQError):
        tq.kv_attention(cache, *args, **bad)
    out, lse = tq.kv_attention(cache, *args, return_lse=True)
    check_attention(b, q64, host(out.double()), host(lse), [1, 1], "f32", 0.125, 0)


# ---- a run of them ------------------------------------------------------------------------------------

def test_decode_steps_captured():
    """Steps of a small server: plan, append, attention, with a request that ends, one that joins
    and prompts in the first step; eager, and as one captured graph replayed with other lengths,
    against the plain form that keeps every key and value."""
    _case("steps")
    g = np.random.default_rng(14)
    kv, G, dim, page, rows, R, mb, pages = 2, 4, 64, 16, 40, 5, 8, 24
    lay = kv_ref.Layout(kv, dim, page)
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    steps = [[9, 20, 0, 3, 0], [1, 1, 0, 1, 14], [1, 1, 33, 1, 1], [1, -1, 1, 1, 1], [1, 6, 1, 0, 1], [1, 1, 1, 1, 1]]
    inputs = [rounded(g.standard_normal((rows, kv * G + 2 * kv, dim)), "bf16") for _ in steps]

    cache = tq.KvCache(kv, dim, page, pages=pages)
    cache.data.fill_(0xFF)
    rope = tq.Rope(dev(inv))
    table, free = i32(np.full((R, mb), -1)), i32(g.permutation(pages))
    length, count, new = i32([0] * R), i32([pages]), i32([0] * R)
    x = torch.zeros((rows, kv * G + 2 * kv, dim), dtype=torch.bfloat16, device="cuda:0")
    q, k, v = x.split([kv * G, kv, kv], dim=1)

    def step():
        p = tq.kv_plan(cache, length, new, table, rows, free, count)
        qt = tq.kv_append(cache, k, v, p["slots"], q=q, rope=rope, positions=p["positions"])
        out, lse = tq.kv_attention(cache, qt, table, p["seq_len"], p["cu_new"], return_lse=True)
        length.copy_(p["seq_len"])
        count.copy_(p["free_count"])
        return p, qt, out, lse

    def run(call):
        """All steps by call(); the numbers of each."""
        table.fill_(-1)
        free.copy_(first_free)
        length.zero_()
        count.fill_(pages)
        seen = []
        for n, (xi, _) in zip(steps, inputs):
            new.copy_(i32(n))
            x.copy_(xi)
            p, qt, out, lse = call()
            torch.cuda.synchronize()
            torch.ones(1000, device="cuda:0").sum()  # eager work between replays
            seen.append((host(p["status"])[0], host(p["seq_len"]), host(p["cu_new"]), host(qt.double()), host(out.double()), host(lse)))
        return seen

    first_free = free.clone()
    eager = run(step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()

    def replay():
        graph.replay()
        return held

    for again in range(3):
        for a, b in zip(eager, run(replay)):
            n = a[2][-1]
            assert a[0] == b[0] == 0 and np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2])
            for i in (3, 4, 5):
                assert np.array_equal(a[i][:n], b[i][:n])

    # the plain form: every request's rounded keys and values in a list
    held_k, held_v, lens = [[] for _ in range(R)], [[] for _ in range(R)], [0] * R
    scratch = np.zeros(lay.page_bytes, np.uint8)
    for n, (_, x64), (_, seq, cu, qt, out, lse) in zip(steps, inputs, eager):
        row = 0
        for r in range(R):
            if n[r] < 0:
                held_k[r], held_v[r], lens[r] = [], [], 0
            for _ in range(max(n[r], 0)):
                turned = kv_ref.turn(x64[row:row + 1, :kv * G + kv], np.array([[lens[r]]]), inv, [32], False)
                tol = torch.finfo(torch.bfloat16).eps / 2 * (1 + 2.0**-20) * np.abs(turned[0, :kv * G]) + 2.0**-133
                tol = tol + 4 * 2.0**-24 * 2 * np.abs(x64[row, :kv * G]).max()  # turned in fp32
                assert (np.abs(qt[row] - turned[0, :kv * G]) <= tol).all()
                kv_ref.write(scratch, lay, [3], turned[:, kv * G:].astype(np.float32), x64[row:row + 1, kv * G + kv:].astype(np.float32))
                a, b = kv_ref.read(scratch, lay, [3])
                held_k[r].append(a[0])
                held_v[r].append(b[0])
                lens[r] += 1
                row += 1
        assert list(seq) == lens and cu[-1] == row
        b = Batch.__new__(Batch)
        b.lay, b.lens = lay, lens
        b.rows = lambda r: (np.array(held_k[r]).reshape(-1, kv, dim), np.array(held_v[r]).reshape(-1, kv, dim))
        check_attention(b, qt[:row], out, lse, [max(m, 0) for m in n], "bf16", dim**-0.5, 0)


def test_projections_around_the_attention():
    """A decode step's attention part over Q4_K weights: q|k|v in one product, append, attention,
    the o projection; against the oracle's products and the plain form, stage by stage."""
    import oracle
    import synth
    from tests.gpu_util import assert_product_close

    _case("projections")
    hidden, kv, G, dim, page, T = 512, 2, 2, 128, 16, 3
    g = synth.rng(21, "kv-layer")
    shapes = {"q": (kv * G * dim, hidden), "k": (kv * dim, hidden), "v": (kv * dim, hidden), "o": (hidden, kv * G * dim)}
    w = {n: synth.blob("q4_k", synth.rng(21, "kv-layer", n), *s) for n, s in shapes.items()}
    wd = {n: dev(b) for n, b in w.items()}
    x = synth.normal_f32(g, (T, hidden)) * np.float32(0.01)
    lens = [40, 17, 1]
    b = Batch(np.random.default_rng(3), kv, dim, page, lens)
    cache = cache_of(b.data, b.lay, page)
    inv = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    q, k, v = tq.gemv_multi("q4_k", [wd[n] for n in "qkv"], [shapes[n][0] for n in "qkv"], hidden, dev(x))
    last = np.array([n - 1 for n in lens])
    slots = [int(b.slots(r)[-1]) for r in range(T)]
    qt = tq.kv_append(cache, k.view(T, kv, dim), v.view(T, kv, dim), i32(slots), q=q.view(T, kv * G, dim),
                      rope=tq.Rope(dev(inv)), positions=i32(last))
    out, lse = tq.kv_attention(cache, qt, i32(b.table), i32(lens), i32([0, 1, 2, 3]), return_lse=True)
    y = tq.gemv("q4_k", wd["o"], *shapes["o"], out.view(T, -1))
    for n, got in zip("qkv", (q, k, v)):
        ref, mag = oracle.gemv("q4_k", w[n], *shapes[n], x)
        assert_product_close(host(got), ref, mag, what=n)
    turned = kv_ref.turn(np.concatenate([host(q).reshape(T, -1, dim), host(k).reshape(T, -1, dim)], 1), last[None], inv, [64], False)
    kv_ref.write(b.data, b.lay, slots, turned[:, kv * G:].astype(np.float32), host(v).reshape(T, kv, dim))
    assert np.array_equal(host(cache.data).ravel(), b.data)
    check_attention(b, host(qt.double()), host(out.double()), host(lse), [1] * T, "f32", dim**-0.5, 0)
    ref, mag = oracle.gemv("q4_k", w["o"], *shapes["o"], host(out).reshape(T, -1))
    assert_product_close(host(y), ref, mag, what="o")
