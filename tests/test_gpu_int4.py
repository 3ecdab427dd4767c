"""The 4-bit cache on the GPU: rows written to it, its pages widened and copied,
decode attention over it.

Tolerances.  Written bytes and widened values are compared bit for bit: both are
defined in fp32 arithmetic.  Decode: the weights carry 2^-22 (a hi + lo pair),
2^-22 (the exponential's instruction) and the fp32 rounding of an exponent of at
most about 64, 4 roundings of 2^-24 * 64 = 2^-16; so a weight is off by 2^-15.5
at most, and an output, a mean of values of magnitude vmax with such weights, by
2 * 2^-15.5 * vmax < 5e-5 vmax.  lse: the same 2^-15.5 plus its own rounding,
5e-5 absolute.
"""
import math

import pytest
import torch

import int4_reference as ref
from paged_kv_attention_14_gb300 import binding as pa
from paged_kv_attention_14_gb300.step import GraphedStep, MixedStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
ACT = {pa.PA_KV_INT4: torch.bfloat16, pa.PA_KV_INT4_F16: torch.float16}
TOL = 5e-5


def _rows(T, hkv, d, act, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    centre = torch.randn((hkv, d), generator=g)
    return ((torch.randn((T, hkv, d), generator=g) + 2 * centre) * scale).to(act)


@pytest.mark.parametrize("kind", [pa.PA_KV_INT4, pa.PA_KV_INT4_F16])
@pytest.mark.parametrize("T,hkv,d", [(1, 1, 64), (3, 2, 64), (33, 8, 128), (257, 3, 128), (16, 2, 128)])
def test_written_bytes(kind, T, hkv, d):
    act = ACT[kind]
    k, v = _rows(T, hkv, d, act, T), _rows(T, hkv, d, act, T + 1, 0.01)
    k[0, 0] = 1.25                   # a group whose dims are all alike
    if T > 3:
        k[1, 0, 3] = float("nan")
        k[2, 0, 5] = float("inf")
        v[1, 1, d - 1] = -float("inf")
        v[3, 0] = 0
        v[2, 0, :64] = 3e-7          # below fp16's normal range (and bf16's spacing around it)
        v[2, 0, 7] = 5e-7
    blocks = T // 16 + 3
    perm = torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(T))[:T].to(torch.int64)
    if T > 16:
        perm[T // 2] = -1
        perm[T - 1] = -5
    base = torch.randint(0, 256, (blocks, hkv, 9 * d), dtype=torch.uint8)
    desc = pa.make_desc(blocks, hkv, hkv, d, kind)
    kc, vc = base.to(DEV), base.flip(0).contiguous().to(DEV)
    pa.pa_cache_write(desc, k.to(DEV), v.to(DEV), kc, vc, perm.to(DEV))
    for x, got, want in ((k, kc, base.clone()), (v, vc, base.flip(0).contiguous())):
        n, s, m = ref.quantise(x)
        tile = ref.pack(n[:, :, None].expand(-1, -1, 16, -1), s[:, :, None].expand(-1, -1, 16, -1),
                        m[:, :, None].expand(-1, -1, 16, -1))
        for i, slot in enumerate(perm.tolist()):
            if slot < 0:
                continue
            b, o = slot // 16, slot % 16
            c, p = slice(o * d // 2, (o + 1) * d // 2), slice(8 * d + o * d // 16, 8 * d + (o + 1) * d // 16)
            want[b, :, c], want[b, :, p] = tile[i, :, c], tile[i, :, p]
        assert torch.equal(got.cpu(), want)


def test_write_reports_values_past_fp16_and_bad_slots():
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(2, 1, 1, 64, pa.PA_KV_INT4, error_word=word, check_indices=True)
    kc, vc = pa.int4_cache(2, 1, 64), pa.int4_cache(2, 1, 64)
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    pa.pa_cache_write(desc, x, x, kc, vc, torch.tensor([3], device=DEV))
    assert int(word) == 0
    y = x.clone()
    y[0, 0, 5] = -1e6
    pa.pa_cache_write(desc, x, y, kc, vc, torch.tensor([4], device=DEV))
    assert int(word) == pa.PA_DEVERR_FP16_RANGE
    assert ref.rows_of(vc.cpu(), 64)[0, 0, 4].isnan().all() and not ref.rows_of(kc.cpu(), 64)[0, 0].isnan().any()
    word.zero_()
    before = kc.clone()
    pa.pa_cache_write(desc, x, x, kc, vc, torch.tensor([32], device=DEV))
    assert int(word) == pa.PA_DEVERR_BAD_INDEX and torch.equal(kc, before)


@pytest.mark.parametrize("kind", [pa.PA_KV_INT4, pa.PA_KV_INT4_F16])
@pytest.mark.parametrize("hkv,d,pairs", [(1, 64, 1), (2, 128, 5), (8, 128, 700), (3, 64, 33)])
def test_widened_pages(kind, hkv, d, pairs):
    act = ACT[kind]
    x = _rows(pairs * 16, hkv, d, act, pairs).view(pairs, 16, hkv, d).transpose(1, 2).contiguous()
    x[0, 0, 0, 0] = float("nan")
    kc, vc = ref.cache_of(x), ref.cache_of(x.flip(0).contiguous() * 0.125)
    g = torch.Generator().manual_seed(pairs)
    src = torch.randint(0, pairs, (pairs,), generator=g, dtype=torch.int32)  # repeats among them
    dst = torch.randperm(pairs + 2, generator=g)[:pairs].to(torch.int32)
    ko = torch.full((pairs + 2, hkv, 16, d), 7.0, dtype=act, device=DEV)
    vo = torch.full_like(ko, 9.0)
    desc = pa.make_desc(pairs, hkv, hkv, d, kind)
    pa.pa_widen_blocks(desc, kc.to(DEV), vc.to(DEV), src.to(DEV), ko, vo, dst.to(DEV))
    for got, cache, fill in ((ko, kc, 7.0), (vo, vc, 9.0)):
        want = torch.full(got.shape, fill, dtype=act)
        want[dst.long()] = ref.rows_of(cache, d)[src.long()].float().to(act)  # s n + m in fp32, rounded once more
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(got.cpu().nan_to_num(0.0), want.nan_to_num(0.0))


def test_widen_skips_and_reports_bad_pages():
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(3, 2, 2, 64, pa.PA_KV_INT4, error_word=word, check_indices=True)
    kc = ref.cache_of(_rows(48, 2, 64, torch.bfloat16, 0).view(3, 16, 2, 64).transpose(1, 2)).to(DEV)
    out = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for src, dst in ((3, 0), (-1, 0), (0, 2), (0, -1)):
        word.zero_()
        pa.pa_widen_blocks(desc, kc, kc, i32(src, 1), out, out.clone(), i32(dst, 1))
        assert int(word) == pa.PA_DEVERR_BAD_INDEX
        assert (out[0] == 0).all() and (out[1] != 0).any()


def test_copied_pages():
    kc = torch.randint(0, 256, (7, 3, 9 * 128), dtype=torch.uint8, device=DEV)
    vc = torch.randint(0, 256, (7, 3, 9 * 128), dtype=torch.uint8, device=DEV)
    want = kc.clone(), vc.clone()
    desc = pa.make_desc(7, 3, 6, 128, pa.PA_KV_INT4)
    pa.pa_copy_blocks(desc, kc, vc, torch.tensor([1, 4], dtype=torch.int32, device=DEV),
                      torch.tensor([6, 0], dtype=torch.int32, device=DEV))
    for got, w in ((kc, want[0]), (vc, want[1])):
        w[6], w[0] = w[1].clone(), w[4].clone()
        assert torch.equal(got, w)


# ------------------------------------------------------------------- decode

class Batch:
    """A batch over a shuffled pool whose other rows (free pages, the rows behind a
    sequence's end) read as NaN."""

    def __init__(self, lens, hq, hkv, d, kind, seed=0, kscale=1.0, vscale=1.0, qscale=1.0, **desc):
        g = torch.Generator().manual_seed(seed)
        act = ACT[kind]
        self.d, self.kind = d, kind
        need = [(x + 15) // 16 for x in lens]
        nb = sum(need) + 3
        ids = torch.randperm(nb, generator=g)
        width = max(1, max(need)) + 1
        self.tables = torch.full((len(lens), width), -1, dtype=torch.int32)
        x = [torch.randn((nb, hkv, 16, d), generator=g) for _ in range(2)]
        self.kc, self.vc = ref.cache_of((x[0] * kscale).to(act)), ref.cache_of((x[1] * vscale).to(act))
        at = 0
        for i, n in enumerate(need):
            self.tables[i, :n] = ids[at:at + n].to(torch.int32)
            at += n
            if lens[i] % 16:
                for c in (self.kc, self.vc):
                    ref.poison(c, d, int(ids[at - 1]), slice(lens[i] % 16, 16))
        for b in ids[at:].tolist():
            for c in (self.kc, self.vc):
                ref.poison(c, d, b, slice(0, 16))
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.q = (torch.randn((len(lens), hq, d), generator=g) * qscale).to(act)
        self.scale = 1.0 / math.sqrt(d)
        self.vmax = float(ref.rows_of(self.vc, d).nan_to_num(0.0).abs().max())
        self.window, self.chunk = desc.get("sliding_window", 0), desc.get("attention_chunk", 0)
        self.word = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.desc = pa.make_desc(nb, hkv, hq, d, kind, error_word=self.word, **desc)
        self.dev = {n: getattr(self, n).to(DEV) for n in ("kc", "vc", "tables", "lens", "q")}
        self.out = torch.full(self.q.shape, float("nan"), device=DEV)
        self.lse = torch.full(self.q.shape[:2], float("nan"), device=DEV)
        self.ws = pa.decode_workspace(self.desc, len(lens), int(max(lens)))

    def run(self, call=None, **kw):
        x = self.dev
        pa.pa_decode(self.desc, self.out, x["q"], x["kc"], x["vc"], x["tables"], x["lens"], int(self.lens.max()),
                     self.scale, self.ws, lse=self.lse, **kw)

    def want(self):
        return ref.decode(self.q, self.kc, self.vc, self.tables, self.lens, self.scale, self.window, self.chunk)

    def check(self):
        out, lse = self.want()
        torch.testing.assert_close(self.out.cpu().double(), out, rtol=0, atol=TOL * self.vmax)
        torch.testing.assert_close(self.lse.cpu().double(), lse, rtol=0, atol=TOL)
        assert int(self.word) == 0 and int(self.ws[:256].sum()) == 0


HEADS = [(4, 2, 64), (32, 8, 128), (5, 5, 128), (16, 1, 128), (9, 1, 64), (12, 2, 128), (16, 2, 64), (1, 1, 64)]


@pytest.mark.parametrize("kind", [pa.PA_KV_INT4, pa.PA_KV_INT4_F16])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens", [[1], [0, 1, 7, 16, 33, 0], [15, 17, 31, 32, 48, 64, 65, 257], [1000, 3, 0, 511]])
def test_decode(kind, hq, hkv, d, lens):
    b = Batch(lens, hq, hkv, d, kind, seed=len(lens))
    b.run()
    b.check()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("lens", [[40001], [20000, 1, 9000], [2500] * 12])
def test_decode_joins_the_pieces_of_long_sequences(hq, hkv, d, lens):
    b = Batch(lens, hq, hkv, d, pa.PA_KV_INT4, seed=3)
    b.run()
    b.check()
    first = b.out.clone(), b.lse.clone()
    for _ in range(3):  # the join's order is the pieces', not the warps'
        b.out.fill_(float("nan"))
        b.run()
        assert torch.equal(b.out, first[0]) and torch.equal(b.lse, first[1])


def test_decode_of_many_sequences():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 70, (1500,), generator=g).tolist()
    lens[700:760] = [0] * 60
    b = Batch(lens, 8, 2, 64, pa.PA_KV_INT4, seed=5)
    b.run()
    b.check()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (3, 1, 64), (16, 1, 128), (10, 2, 64)])
@pytest.mark.parametrize("lens", [[1024] * 24, [1025, 0] + [1024] * 9, [0, 0], [0] * 300 + [700] + [0] * 500 + [33, 0],
                                  list(range(400)), [64] * 152 + [0], [1] * 513])
def test_decode_around_what_is_dealt_whole(hq, hkv, d, lens):
    b = Batch(lens, hq, hkv, d, pa.PA_KV_INT4, seed=6)
    b.run()
    b.check()
    first = b.out.clone()
    b.run()
    assert torch.equal(b.out, first)


@pytest.mark.parametrize("local", [dict(sliding_window=1), dict(sliding_window=5), dict(sliding_window=100),
                                   dict(attention_chunk=64), dict(attention_chunk=48, sliding_window=20)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 1, 64)])
def test_decode_of_local_layers(local, hq, hkv, d):
    lens = [1, 4, 5, 6, 63, 64, 65, 99, 100, 101, 129, 1000]
    b = Batch(lens, hq, hkv, d, pa.PA_KV_INT4, seed=7, **local)
    for i, L in enumerate(lens):  # pages before the first key may hold anything
        lo = ref.first_key(L - 1, b.window, b.chunk)
        for e in range(lo // 16):
            b.dev["tables"][i, e] = b.desc.num_blocks - 1
            for c in ("kc", "vc"):
                ref.poison(b.dev[c], d, int(b.tables[i, e]), slice(0, 16))
    b.run()
    b.check()


@pytest.mark.parametrize("kscale,vscale,qscale", [(1e-3, 1e-4, 1.0), (30.0, 300.0, 0.03), (1.0, 1e-6, 1e-6),
                                                  (1e-4, 1.0, 1e4), (0.0, 0.0, 1.0)])
@pytest.mark.parametrize("kind", [pa.PA_KV_INT4, pa.PA_KV_INT4_F16])
def test_decode_of_small_and_large_values(kscale, vscale, qscale, kind):
    if kind == pa.PA_KV_INT4_F16 and qscale < 1e-5:
        qscale = 1e-3
    b = Batch([700, 33, 16], 8, 2, 128, kind, seed=11, kscale=kscale, vscale=vscale, qscale=qscale)
    b.run()
    b.check()


def test_decode_of_values_that_grow_along_the_sequence():
    # the scales pass the first blocks' by far, and the scores rise
    b = Batch([600, 900], 8, 2, 128, pa.PA_KV_INT4, seed=12)
    d = 128
    for s in range(2):
        for e in range(int(b.lens[s] + 15) // 16):
            f = 2.0 ** (e // 4 - 8)
            for c in (b.kc, b.vc):
                pairs = c[int(b.tables[s, e]), :, 8 * d:].contiguous().view(torch.float16)
                c[int(b.tables[s, e]), :, 8 * d:] = (pairs.float() * (f if c is b.vc else 1 + e / 8)).half().view(torch.uint8)
    b.dev["kc"], b.dev["vc"] = b.kc.to(DEV), b.vc.to(DEV)
    b.vmax = float(ref.rows_of(b.vc, d).nan_to_num(0.0).abs().max())
    b.run()
    out, lse = b.want()
    # scores of magnitude 60 here: the exponent's rounding is 2^-24 * 90 * 4 = 2^-15.5, as derived above
    torch.testing.assert_close(b.out.cpu().double(), out, rtol=0, atol=TOL * b.vmax)
    torch.testing.assert_close(b.lse.cpu().double(), lse, rtol=0, atol=2 * TOL)


def test_a_nan_key_or_value_reaches_its_own_sequence_and_head_only():
    b = Batch([200, 50, 120], 8, 2, 64, pa.PA_KV_INT4, seed=13)
    pairs = b.kc[..., 8 * 64:].unflatten(-1, (16, 4))
    pairs[int(b.tables[1, 2]), 1, 3, 0::2] = 0xFF
    pairs[int(b.tables[1, 2]), 1, 3, 1::2] = 0x7F
    b.dev["kc"] = b.kc.to(DEV)
    b.run()
    got = b.out.cpu()
    assert got[1, 4:].isnan().all() and not got[1, :4].isnan().any()
    assert not got[0].isnan().any() and not got[2].isnan().any()


def test_decode_on_another_stream_captured_and_with_checked_indices():
    b = Batch([300, 0, 17], 8, 2, 128, pa.PA_KV_INT4, seed=14, check_indices=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    b.check()
    graph = GraphedStep(b.run)
    b.out.fill_(0)
    # the replay sees new lengths and queries
    b.lens = torch.tensor([5, 290, 0], dtype=torch.int32)
    b.tables = b.tables[[2, 0, 1]].contiguous()
    b.dev["lens"].copy_(b.lens)
    b.dev["tables"].copy_(b.tables)
    graph()
    # (rows 5..15 of the first sequence's page are its own old rows, finite)
    b.check()
    b.dev["tables"][1, 3] = 10 ** 6
    b.run()
    assert int(b.word) == pa.PA_DEVERR_BAD_INDEX


def test_decode_static_and_pinned_outputs():
    b = Batch([300, 4000, 17], 8, 2, 128, pa.PA_KV_INT4, seed=15)
    x = b.dev
    out, lse = torch.zeros(b.q.shape).pin_memory(), torch.zeros(b.q.shape[:2]).pin_memory()
    pa.pa_decode(b.desc, out, x["q"], x["kc"], x["vc"], x["tables"], x["lens"], 4000, b.scale, b.ws, lse=lse)
    torch.cuda.synchronize()
    b.out.copy_(out)
    b.lse.copy_(lse)
    b.check()
    b.out.fill_(0)
    for _ in range(2):
        pa.pa_decode_static(b.desc, b.out, x["q"], x["kc"], x["vc"], x["tables"], x["lens"], 4000, b.scale, lse=b.lse)
        b.check()


def test_a_cache_past_32_bits():
    """Rows whose bytes lie past 2^32 are written, widened and attended where they are."""
    hkv, d, nb = 8, 128, 480_000  # 4.4 GB each
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 10 GB")
    desc = pa.make_desc(nb, hkv, hkv, d, pa.PA_KV_INT4, check_indices=True)
    kc, vc = pa.int4_cache(nb, hkv, d), pa.int4_cache(nb, hkv, d)
    pages = [nb - 1, 3, nb - 7]
    small = pa.make_desc(3, hkv, hkv, d, pa.PA_KV_INT4)
    ks, vs = pa.int4_cache(3, hkv, d), pa.int4_cache(3, hkv, d)
    T = 45
    k, v = [x.to(DEV) for x in (_rows(T, hkv, d, torch.bfloat16, 1), _rows(T, hkv, d, torch.bfloat16, 2))]
    i = torch.arange(T, device=DEV)
    at = torch.tensor(pages, device=DEV)
    pa.pa_cache_write(desc, k, v, kc, vc, at[i // 16] * 16 + i % 16)
    pa.pa_cache_write(small, k, v, ks, vs, i)
    for p, q in enumerate(pages):
        assert torch.equal(kc[q], ks[p]) and torch.equal(vc[q], vs[p])
    q = torch.randn((1, hkv, d), device=DEV).to(torch.bfloat16)
    outs = []
    for de, c, tab in ((desc, (kc, vc), pages), (small, (ks, vs), [0, 1, 2])):
        out = torch.zeros((1, hkv, d), device=DEV)
        pa.pa_decode(de, out, q, *c, torch.tensor([tab], dtype=torch.int32, device=DEV),
                     torch.tensor([T], dtype=torch.int32, device=DEV), T, 0.1, pa.decode_workspace(de, 1, T))
        wide = torch.zeros((2, 3, hkv, 16, d), dtype=torch.bfloat16, device=DEV)
        pa.pa_widen_blocks(de, *c, torch.tensor(tab, dtype=torch.int32, device=DEV), wide[0], wide[1],
                           torch.arange(3, dtype=torch.int32, device=DEV))
        outs.append((out, wide))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_two_decodes_at_once():
    a, b = Batch([3000, 70, 5], 8, 2, 128, pa.PA_KV_INT4, seed=17), Batch([900] * 20, 16, 1, 64, pa.PA_KV_INT4_F16, seed=18)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st in zip((a, b), streams):
            x.run(stream=st)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_steps_over_a_4_bit_cache():
    """A layer's tokens rotated, written, attended; a chunk behind them over the widened pages."""
    hq, hkv, d, steps, n = 8, 2, 64, 20, 3
    b = Batch([40, 16, 7], hq, hkv, d, pa.PA_KV_INT4, seed=16)
    nb = 64
    kc, vc = pa.int4_cache(nb, hkv, d), pa.int4_cache(nb, hkv, d)
    kc[:b.kc.shape[0]], vc[:b.vc.shape[0]] = b.dev["kc"], b.dev["vc"]
    desc = pa.make_desc(nb, hkv, hq, d, pa.PA_KV_INT4)
    tables = torch.full((n, 8), -1, dtype=torch.int32)
    tables[:, :b.tables.shape[1]] = b.tables
    free = iter(range(b.kc.shape[0], nb))
    lens = b.lens.clone()
    out = torch.zeros((n, hq, d), device=DEV)
    ws = pa.decode_workspace(desc, n, 128)
    step = MixedStep(desc, kc, vc, b.scale, decode_out=out, workspace=ws, max_context_len_decode=128, mode="serial",
                     decode_append=True)
    rope = pa.make_rope(pa.rope_table(256, d))
    g = torch.Generator(device=DEV).manual_seed(1)
    for _ in range(steps):
        qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device=DEV).to(torch.bfloat16)
        slots = []
        for s in range(n):
            e = int(lens[s]) // 16
            if tables[s, e] < 0:
                tables[s, e] = next(free)
            slots.append(int(tables[s, e]) * 16 + int(lens[s]) % 16)
        pos = lens.to(DEV)
        lens += 1
        q = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV)
        k = torch.empty((n, hkv, d), dtype=torch.bfloat16, device=DEV)
        pa.pa_qk_norm_rope(desc, rope, q, k, qkv[:, :hq], qkv[:, hq:hq + hkv], pos)
        step(k, qkv[:, hq + hkv:].contiguous(), torch.tensor(slots, device=DEV),
             dec_args=(q, tables.to(DEV), lens.to(DEV)))
        want, _ = ref.decode(q.cpu(), kc.cpu(), vc.cpu(), tables, lens, b.scale)
        torch.testing.assert_close(out.cpu().double(), want, rtol=0, atol=TOL * 8)
    # a chunk of 24 tokens behind the first sequence: its pages widened, the chunk's rows beside them
    L, c = int(lens[0]), 24
    pages = (L + 15) // 16
    wide = (L + c + 15) // 16
    d16 = pa.make_desc(wide, hkv, hq, d, pa.PA_KV_BF16)
    k16 = torch.zeros((wide, hkv, 16, d), dtype=torch.bfloat16, device=DEV)
    v16 = torch.zeros_like(k16)
    ids = torch.arange(wide, dtype=torch.int32, device=DEV)
    pa.pa_widen_blocks(desc, kc, vc, tables[0, :pages].contiguous().to(DEV), k16, v16, ids[:pages])
    q, k, v = [torch.randn((c, h, d), generator=g, device=DEV).to(torch.bfloat16) for h in (hq, hkv, hkv)]
    pa.pa_cache_write(d16, k, v, k16, v16, torch.arange(L, L + c, device=DEV))
    got = torch.zeros((c, hq, d), device=DEV)
    pa.pa_prefill_chunk(d16, got, q, torch.tensor([0, c], dtype=torch.int32, device=DEV), k16, v16, ids[None],
                        torch.tensor([L + c], dtype=torch.int32, device=DEV), c, L + c, b.scale)
    at = tables[0, :pages].long()
    old = [ref.rows_of(x.cpu()[at], d).permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :L] for x in (kc, vc)]
    kk, vv = [torch.cat([o.to(torch.bfloat16).double(), x.cpu().double().transpose(0, 1)], 1)
              for o, x in zip(old, (k, v))]
    x = (q.cpu().double().transpose(0, 1).view(hkv, hq // hkv, c, d) @ kk[:, None].transpose(-1, -2)) * b.scale
    x = x.masked_fill(torch.arange(L + c)[None, :] > torch.arange(L, L + c)[:, None], -math.inf)
    want = (torch.softmax(x, -1) @ vv[:, None]).reshape(hq, c, d).transpose(0, 1)
    torch.testing.assert_close(got.cpu().double(), want, rtol=0, atol=2e-3)  # pa_prefill_chunk's tolerance


def test_prompts_then_steps_over_a_4_bit_cache():
    """Prompts attended on their own rows and written to a 4-bit cache, then decode steps over it, with the prompts'
    call and a step each in a graph."""
    hq, hkv, d, lens = 8, 2, 128, [37, 100, 16]
    nb, n, T = 40, len(lens), sum(lens)
    desc = pa.make_desc(nb, hkv, hq, d, pa.PA_KV_INT4)
    kc, vc = pa.int4_cache(nb, hkv, d), pa.int4_cache(nb, hkv, d)
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(2))[:n * 10].view(n, 10).to(torch.int32)
    slots = torch.cat([tables[s].long()[torch.arange(L) // 16] * 16 + torch.arange(L) % 16 for s, L in enumerate(lens)])
    g = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn((T, hq + 2 * hkv, d), generator=g, device=DEV).to(torch.bfloat16)
    v = qkv[:, hq + hkv:].contiguous()
    rope = pa.make_rope(pa.rope_table(256, d))
    pos = torch.cat([torch.arange(L) for L in lens]).to(torch.int32).to(DEV)
    starts = torch.tensor([0, 37, 137, 153], dtype=torch.int32, device=DEV)
    q_rot = torch.empty((T, hq, d), dtype=torch.bfloat16, device=DEV)
    k_rot = torch.empty((T, hkv, d), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q_rot)
    dec = torch.zeros((n, hq, d), device=DEV)
    scale = 1 / math.sqrt(d)
    step = MixedStep(desc, kc, vc, scale, decode_out=dec, workspace=pa.decode_workspace(desc, n, 160),
                     max_context_len_decode=160, mode="serial")
    dslots = slots.to(DEV)
    graph = GraphedStep(lambda: step.prompts(out, qkv[:, :hq], qkv[:, hq:hq + hkv], v, starts, 100, dslots, rope=rope,
                                             positions=pos, q_rot=q_rot, k_rot=k_rot))
    kc.zero_()
    vc.zero_()
    graph()
    at = 0
    for L in lens:  # the rotated rows' own attention
        x = q_rot[at:at + L].cpu().double().transpose(0, 1).view(hkv, hq // hkv, L, d)
        x = x @ k_rot[at:at + L].cpu().double().transpose(0, 1)[:, None].transpose(-1, -2) * scale
        p = torch.softmax(x.masked_fill(torch.ones(L, L).triu(1).bool(), -math.inf), -1)
        vv = v[at:at + L].cpu().double().transpose(0, 1)[:, None]
        want, size = [(p @ y).reshape(hq, L, d).transpose(0, 1) for y in (vv, vv.abs())]
        off = (out[at:at + L].cpu().double() - want).abs()
        assert (off <= 2.0 ** -8 * (size + want.abs()) + 2.0 ** -15 * size).all()
        at += L
    # the rows in the cache, and steps behind them
    stored = ref.rows_of(kc.cpu(), d)[slots // 16, :, slots % 16]
    codes, s, m = ref.quantise(k_rot.cpu())
    assert torch.equal(stored, (codes.double().unflatten(-1, (-1, 64)) * s.double()[..., None] +
                                m.double()[..., None]).flatten(-2))
    now = torch.tensor(lens, dtype=torch.int32)
    bufs = dict(q=q_rot[:n].clone(), k=k_rot[:n].clone(), v=v[:n].clone(), slots=torch.zeros(n, dtype=torch.int64, device=DEV),
                tables=tables.to(DEV), lens=now.to(DEV))
    one = GraphedStep(lambda: step(bufs["k"], bufs["v"], bufs["slots"],
                                   dec_args=(bufs["q"], bufs["tables"], bufs["lens"])))
    for i in range(5):
        bufs["slots"].copy_(tables[torch.arange(n), now.long() // 16].long() * 16 + now.long() % 16)
        now += 1
        bufs["lens"].copy_(now)
        for b in ("q", "k", "v"):
            bufs[b].copy_(torch.randn(bufs[b].shape, generator=g, device=DEV))
        one()
        want, _ = ref.decode(bufs["q"].cpu(), kc.cpu(), vc.cpu(), tables, now, scale)
        vmax = float(ref.rows_of(vc.cpu(), d).abs().max())
        torch.testing.assert_close(dec.cpu().double(), want, rtol=0, atol=TOL * vmax)
