"""pa_qk_norm_rope and pa_rope_cache_write against their definition in 64 bits.

Tolerance: one rounding of the result (half a step: eps / 2 of its type,
relative to the value) plus the fp32 arithmetic before it.  The mean square
is a sum of at most 128 products in a tree of 16 + 3 additions, rsqrt is
within 2 ulp, and each result is a difference of two products: fewer than 32
roundings of 2^-24 each, relative to |y_i| + |y_j|, so 2^-19 (|y_i| + |y_j|).
fp16 results below 2^-14 are subnormal: their steps are 2^-24 whatever the
value, so a rounding there is off by up to 2^-25 (bf16 has fp32's exponents;
its subnormals lie below 1e-38).
"""
import numpy as np
import pytest
import torch

from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300.step import GraphedStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}
FP8 = {B.PA_KV_FP8_E4M3: (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10),
       B.PA_KV_FP8_E5M2: (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}
MAXP = 5000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())


class Case:
    def __init__(self, T, hq, hkv, D, rd, inter, norm, kv=B.PA_KV_BF16, seed=0, packed=True, blocks=None, **desc):
        g = torch.Generator().manual_seed(seed + 7 * T + D)
        self.T, self.hq, self.hkv, self.D, self.rd, self.inter, self.kv = T, hq, hkv, D, rd, inter, kv
        self.act = torch.float16 if kv == B.PA_KV_F16 else torch.bfloat16
        x = torch.randn(T, (hq + 2 * hkv) * D, generator=g).to(self.act).to(DEV)
        cut = lambda lo, n: x[:, lo * D:(lo + n) * D].view(T, n, D)  # noqa: E731
        self.q, self.k, self.v = cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv)
        if not packed:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(self.act).to(DEV)  # noqa: E731
        self.qw = w() if "q" in norm else None
        self.kw = w() if "k" in norm else None
        self.table = B.rope_table(MAXP, rd, base=1e6, device=DEV)
        self.pos = torch.randint(0, MAXP, (T,), generator=g).to(torch.int32).to(DEV)
        if T > 2:
            self.pos[0], self.pos[1] = 0, MAXP - 1
        self.eps = 1e-6
        self.nb = blocks or (T + 15) // 16 + 2
        self.slots = torch.randperm(self.nb * 16, generator=g)[:T].to(DEV)
        self.ks, self.vs = (0.02, 0.03) if kv in FP8 else (0.0, 0.0)
        self.desc = B.make_desc(self.nb, hkv, hq, D, kv, k_scale=self.ks, v_scale=self.vs, **desc)
        self.rope = B.make_rope(self.table, interleaved=inter, q_weight=self.qw, k_weight=self.kw, eps=self.eps)

    def ref(self, x, w):
        """The definition in 64 bits: (result, |y_i| + |y_j| of every element)."""
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + self.eps) * w.double()
        out, mag = y.clone(), y.abs()
        for i in range(self.rd // 2):
            a, b = (2 * i, 2 * i + 1) if self.inter else (i, i + self.rd // 2)
            c = self.table[self.pos.long(), i].double()[:, None]
            s = self.table[self.pos.long(), self.rd // 2 + i].double()[:, None]
            out[..., a] = y[..., a] * c - y[..., b] * s
            out[..., b] = y[..., b] * c + y[..., a] * s
            mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
        return out, mag

    def check(self, got, x, w, what):
        want, mag = self.ref(x, w)
        err = (got.double() - want).abs()
        bound = HALF[got.dtype] * want.abs() + 2.0 ** -19 * mag + TINY[got.dtype]
        bad = err > bound
        assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / bound).max()):.2f} of the bound"

    def outs(self):
        return (torch.full((self.T, self.hq, self.D), float("nan"), dtype=self.act, device=DEV),
                torch.full((self.T, self.hkv, self.D), float("nan"), dtype=self.act, device=DEV))

    def caches(self):
        shape = (self.nb, self.hkv, 16, self.D)
        if self.kv in FP8:
            g = torch.Generator().manual_seed(3)
            c = torch.randint(0, 100, shape, generator=g, dtype=torch.uint8).to(DEV)
            return c, c.flip(0).contiguous()
        c = torch.randn(shape, generator=torch.Generator().manual_seed(3)).to(self.act).to(DEV)
        return c, c.flip(0).contiguous()

    def write(self, kc, vc, q_out, slots=None, **kw):
        B.pa_rope_cache_write(self.desc, self.rope, q_out, self.q if q_out is not None else None, self.k, self.v,
                              self.pos, kc, vc, self.slots if slots is None else slots, **kw)


SHAPES = [  # (T, q heads, kv heads, D, rotary dims)
    (1, 32, 8, 128, 128), (1, 4, 2, 64, 64), (2, 16, 1, 128, 64), (3, 8, 8, 128, 16), (5, 40, 8, 128, 128),
    (7, 3, 1, 64, 32), (33, 32, 8, 64, 64), (130, 4, 4, 128, 112), (517, 5, 1, 64, 48), (1031, 40, 8, 128, 128),
]


@pytest.mark.parametrize("norm", ["qk", "", "q", "k"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("fp16", [False, True])
@pytest.mark.parametrize("T,hq,hkv,D,rd", SHAPES)
def test_norm_rope(T, hq, hkv, D, rd, inter, norm, fp16):
    c = Case(T, hq, hkv, D, rd, inter, norm, B.PA_KV_F16 if fp16 else B.PA_KV_BF16, packed=(T % 2 == 1))
    qo, ko = c.outs()
    B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q, c.k, c.pos)
    c.check(qo, c.q, c.qw, "q")
    c.check(ko, c.k, c.kw, "k")


@pytest.mark.parametrize("norm", ["qk", ""])
@pytest.mark.parametrize("kv", [B.PA_KV_BF16, B.PA_KV_F16, B.PA_KV_FP8_E4M3, B.PA_KV_FP8_E5M2])
@pytest.mark.parametrize("T,hq,hkv,D,rd", SHAPES)
def test_cache_write(T, hq, hkv, D, rd, kv, norm):
    c = Case(T, hq, hkv, D, rd, T % 3 == 0, norm, kv, seed=5)
    slots = c.slots.clone()
    slots[::4] = -1  # padding tokens
    if T == 1:
        slots[0] = 17
    kc0, vc0 = c.caches()
    kc, vc = kc0.clone(), vc0.clone()
    qo, ko = c.outs()
    c.write(kc, vc, qo, slots)
    c.check(qo, c.q, c.qw, "q")
    # the rows the two separate calls write, and nothing else
    B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q, c.k, c.pos)
    kc2, vc2 = kc0.clone(), vc0.clone()
    B.pa_cache_write(c.desc, ko, c.v.contiguous(), kc2, vc2, slots)
    assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
    live = slots >= 0
    blk, off = slots[live] // 16, slots[live] % 16
    if kv not in FP8:
        assert torch.equal(kc.view(torch.int16), kc2.view(torch.int16))
        return
    kind, top, half, tiny = FP8[kv]
    want, mag = c.ref(c.k, c.kw)
    want, mag = want[live] / np.float32(c.ks), mag[live] / np.float32(c.ks)
    got = kc[blk, :, off, :].view(kind).double()
    lim = want.clamp(-top, top)
    # one rounding to the 8-bit type (its subnormals: half the smallest step), the fp32 steps and division before it
    assert ((got - lim).abs() <= half * lim.abs() + tiny + 2.0 ** -18 * mag).all()
    touched = torch.zeros(c.nb, 16, dtype=torch.bool, device=DEV)
    touched[blk, off] = True
    keep = ~touched[:, None, :, None].expand(kc.shape)
    assert torch.equal(kc[keep], kc0[keep])


@pytest.mark.parametrize("kv", [B.PA_KV_BF16, B.PA_KV_F16, B.PA_KV_FP8_E4M3, B.PA_KV_FP8_E5M2])
@pytest.mark.parametrize("T,hq,hkv,D,rd,inter,norm", [
    (2701, 32, 8, 128, 128, False, "qk"), (1803, 40, 8, 128, 64, True, "q"), (5003, 24, 6, 64, 64, False, "k"),
    (700, 128, 8, 128, 16, False, ""), (400, 256, 16, 128, 128, False, "qk")])
def test_many_tokens(T, hq, hkv, D, rd, inter, norm, kv):
    """Batches of 20 MB of rows and more, read through the ring of stages: an
    odd last stage, packed and dense inputs, padding, one token per stage."""
    c = Case(T, hq, hkv, D, rd, inter, norm, kv, seed=21, packed=T % 2 == 1)
    qo, ko = c.outs()
    B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q, c.k, c.pos)
    c.check(qo, c.q, c.qw, "q")
    c.check(ko, c.k, c.kw, "k")
    slots = c.slots.clone()
    slots[::5] = -1
    kc0, vc0 = c.caches()
    kc, vc, kc2, vc2 = kc0.clone(), vc0.clone(), kc0.clone(), vc0.clone()
    q2 = torch.empty_like(qo)
    c.write(kc, vc, q2, slots)
    assert torch.equal(q2, qo)
    # the kernel of few tokens writes the same bits
    for lo in range(0, T, 64):
        part = slice(lo, lo + 64)
        B.pa_rope_cache_write(c.desc, c.rope, q2[part], c.q[part], c.k[part], c.v[part], c.pos[part], kc2, vc2,
                              slots[part])
    assert torch.equal(q2, qo)
    assert torch.equal(kc.view(torch.uint8), kc2.view(torch.uint8))
    assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
    # in place
    q3, k3 = c.q.contiguous().clone(), c.k.contiguous().clone()
    B.pa_qk_norm_rope(c.desc, c.rope, q3, k3, q3, k3, c.pos)
    assert torch.equal(q3, qo) and torch.equal(k3, ko)


def test_many_tokens_checked():
    ew = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = Case(2500, 32, 8, 128, 128, False, "qk", error_word=ew, check_indices=True)
    kc0, vc0 = c.caches()
    kc, vc, qo = kc0.clone(), vc0.clone(), c.outs()[0]
    c.write(kc, vc, qo)
    assert int(ew) == 0
    c.pos[1000], c.pos[2499] = -5, MAXP
    slots = c.slots.clone()
    slots[7] = c.nb * 16 + 3
    kc2, vc2, qo2 = kc0.clone(), vc0.clone(), torch.empty_like(qo)
    c.write(kc2, vc2, qo2, slots)
    assert int(ew) == B.PA_DEVERR_BAD_INDEX
    keep = torch.ones(2500, dtype=torch.bool, device=DEV)
    keep[1000] = keep[2499] = False
    assert torch.equal(qo2[keep], qo[keep])
    keep[7] = False
    at = c.slots[keep]
    assert torch.equal(kc2[at // 16, :, at % 16], kc[at // 16, :, at % 16])
    assert torch.equal(kc2[c.slots[7] // 16, :, c.slots[7] % 16], kc0[c.slots[7] // 16, :, c.slots[7] % 16])


@pytest.mark.parametrize("kv", [B.PA_KV_FP8_E4M3, B.PA_KV_FP8_E5M2])
def test_per_head_scales(kv):
    c = Case(40, 8, 4, 128, 128, False, "qk", kv, seed=9)
    s = torch.tensor([0.01, 0.02, 0.5, 3.0], device=DEV)
    d = B.make_desc(c.nb, 4, 8, 128, kv, k_scales=s, v_scales=s.flip(0).contiguous())
    kc, vc = (torch.zeros(c.nb, 4, 16, 128, dtype=torch.uint8, device=DEV) for _ in range(2))
    B.pa_rope_cache_write(d, c.rope, None, None, c.k, c.v, c.pos, kc, vc, c.slots)
    kind, top, half, tiny = FP8[kv]
    want, mag = c.ref(c.k, c.kw)
    sk = s.double()[None, :, None]
    got = kc[c.slots // 16, :, c.slots % 16, :].view(kind).double()
    lim = (want / sk).clamp(-top, top)
    assert ((got - lim).abs() <= half * lim.abs() + tiny + 2.0 ** -18 * mag / sk).all()
    vw = (c.v.float() / s.flip(0)[None, :, None]).clamp(-top, top)
    assert torch.equal(vc[c.slots // 16, :, c.slots % 16, :], vw.to(kind).view(torch.uint8))


def test_in_place_one_side_and_empty():
    c = Case(37, 8, 2, 128, 128, False, "qk", packed=False)
    q, k = c.q.clone(), c.k.clone()
    B.pa_qk_norm_rope(c.desc, c.rope, q, k, q, k, c.pos)
    c.check(q, c.q, c.qw, "q in place")
    c.check(k, c.k, c.kw, "k in place")
    ko = c.outs()[1]
    B.pa_qk_norm_rope(c.desc, c.rope, None, ko, None, c.k, c.pos)
    assert torch.equal(ko, k)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    B.pa_qk_norm_rope(c.desc, c.rope, None, c.k[:0], None, c.k[:0], none)


def test_a_row_of_nan_or_infinity_stays_in_its_row_and_zeros_stay_zero():
    c = Case(6, 8, 2, 128, 64, False, "qk", packed=False)
    c.q[1, 3, 5] = float("nan")
    c.q[2, 0, 100] = float("inf")
    c.q[3] = 0
    qo, ko = c.outs()
    B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q, c.k, c.pos)
    bad = ~torch.isfinite(qo).all(-1)
    want = torch.zeros(6, 8, dtype=torch.bool, device=DEV)
    want[1, 3] = want[2, 0] = True
    assert torch.equal(bad, want)
    assert (qo[3] == 0).all() and torch.isfinite(ko).all()


def test_large_and_small_magnitudes():
    """The sum of squares holds in fp32 for bf16 values from 1e-15 to 1e15."""
    for f in (1e-15, 1e15):
        c = Case(4, 4, 2, 128, 128, True, "qk", packed=False)
        c.q.mul_(f)
        qo, ko = c.outs()
        B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q, c.k, c.pos)
        c.check(qo, c.q, c.qw, f"q x {f}")


def test_checked_positions_and_slots_are_reported_and_skipped():
    ew = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = Case(8, 8, 2, 128, 128, False, "qk", error_word=ew, check_indices=True)
    good = c.pos.clone()
    kc0, vc0 = c.caches()
    kc, vc = kc0.clone(), vc0.clone()
    qo, ko = c.outs()
    c.write(kc, vc, qo)
    assert int(ew) == 0
    c.pos[3], c.pos[4] = -1, MAXP
    slots = c.slots.clone()
    slots[5] = c.nb * 16
    kc2, vc2 = kc0.clone(), vc0.clone()
    qo2 = torch.empty_like(qo)
    c.write(kc2, vc2, qo2, slots)
    assert int(ew) == B.PA_DEVERR_BAD_INDEX
    rows = [0, 1, 2, 5, 6, 7]
    assert torch.equal(qo2[rows], qo[rows])
    rows = [0, 1, 2, 6, 7]
    at = c.slots[rows]
    assert torch.equal(kc2[at // 16, :, at % 16], kc[at // 16, :, at % 16])
    assert torch.equal(kc2[c.slots[5] // 16, :, c.slots[5] % 16], kc0[c.slots[5] // 16, :, c.slots[5] % 16])
    c.pos.copy_(good)


@pytest.mark.parametrize("tokens", [8, 4096])
def test_padding_positions_take_position_0(tokens):
    """Unchecked positions outside the table (padding tokens') read nothing outside it; both kernels."""
    c = Case(tokens, 32, 8, 128, 128, False, "qk")
    outside = torch.arange(tokens, device=DEV) % 5 == 3
    c.pos[outside] = 0
    want_q, want_k = c.outs()
    B.pa_qk_norm_rope(c.desc, c.rope, want_q, want_k, c.q, c.k, c.pos)
    c.pos[outside] = torch.tensor([-1, MAXP, 2**31 - 1, -2**31], dtype=torch.int32, device=DEV).repeat(tokens)[
        :int(outside.sum())]
    qo, ko = c.outs()
    B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q, c.k, c.pos)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)


def test_other_stream_and_graph_replay():
    c = Case(50, 32, 8, 128, 128, False, "qk", seed=11)
    want_q, _ = c.outs()
    kc0, vc0 = c.caches()
    want_k, want_v = kc0.clone(), vc0.clone()
    c.write(want_k, want_v, want_q)
    torch.cuda.synchronize()
    kc, vc, qo = kc0.clone(), vc0.clone(), c.outs()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.write(kc, vc, qo, stream=side)
    side.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(kc, want_k) and torch.equal(vc, want_v)
    step = GraphedStep(lambda: c.write(kc, vc, qo))
    # the replay reads what the buffers hold then
    c.q.copy_(torch.randn(c.q.shape, device=DEV).to(c.act))
    c.pos.copy_((c.pos + 1) % MAXP)
    step()
    c.check(qo, c.q, c.qw, "replayed q")


def test_misuse_of_the_binding_is_refused():
    c = Case(6, 8, 2, 128, 128, False, "qk", packed=False)
    qo, ko = c.outs()
    with pytest.raises(ValueError, match="must be"):
        B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q[:5], c.k, c.pos)
    with pytest.raises(ValueError, match="contiguous"):
        B.pa_qk_norm_rope(c.desc, c.rope, qo, ko, c.q.transpose(0, 1).contiguous().transpose(0, 1), c.k, c.pos)
    wide = torch.empty(6, 9, 128, dtype=c.act, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        B.pa_qk_norm_rope(c.desc, c.rope, wide[:, :8], ko, c.q, c.k, c.pos)
    with pytest.raises(ValueError, match="head_dim"):
        r = B.make_rope(c.table, q_weight=c.qw.half(), k_weight=c.kw)
        B.pa_qk_norm_rope(c.desc, r, qo, ko, c.q, c.k, c.pos)
    kc, vc = c.caches()
    with pytest.raises(ValueError, match="num_blocks"):
        c.write(kc[:-1], vc, qo)
    with pytest.raises(ValueError, match="one entry"):
        c.write(kc, vc, qo, c.slots[:-1])
    with pytest.raises(ValueError, match="k and v"):
        B.pa_rope_cache_write(c.desc, c.rope, qo, c.q, None, c.v, c.pos, kc, vc, c.slots)
