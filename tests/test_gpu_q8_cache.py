"""The 8-bit paged cache on the GPU, against a plain 64-bit reference: the
append, the attention over it in every schedule, the accumulated block weights
and the eviction, and a run of them together."""
import math

import pytest
import torch

import long_context_indexer_b200 as lci

from . import q8_reference as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def vals(pool):
    return pool.cpu().float().double()


def make_table(B, NB, P, gen):
    return torch.randperm(P, generator=gen)[: B * NB].reshape(B, NB).to(torch.int32).contiguous()


def make_cache(P, H, bs, hd, gen, fill_nan=True):
    c = lci.Q8Cache(P, H, bs, hd, "cuda")
    if fill_nan:
        c.k.view(torch.uint8).fill_(0x7F)
        c.v.view(torch.uint8).fill_(0x7F)
    return c


def filled_cache(B, H, bs, hd, lens, seed, spread=2.0):
    """(cache, table, cpu copies): random codes and scales, NaN codes in slots
    behind each sequence's last token and in pages no sequence holds."""
    g = torch.Generator().manual_seed(seed)
    NB = max(1, -(-max(lens) // bs))
    P = B * NB + 3
    table = make_table(B, NB, P, g)
    cpu = []
    for _ in range(2):
        x = torch.randn(P, H, bs, hd, generator=g)
        scale = torch.exp2((torch.rand(P, H, generator=g) - 0.5) * spread) / 64
        code = (x / scale[:, :, None, None]).clamp(-448, 448).to(E4M3)
        raw = code.view(torch.uint8)
        used = torch.zeros(P, dtype=torch.bool)
        for b, n in enumerate(lens):
            nb = -(-n // bs)
            used[table[b, :nb].long()] = True
            if n % bs:
                raw[int(table[b, nb - 1]), :, n % bs:] = 0x7F
        raw[~used] = 0x7F
        cpu += [code, scale]
    k, ks, v, vs = cpu
    cache = lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs)))
    return cache, table, (k, v, ks, vs)


def random_ids(B, S, NB, topk, gen, hole=0.1):
    ids = torch.full((B, S, topk), -1, dtype=torch.int32)
    for b in range(B):
        for s in range(S):
            pick = torch.randperm(NB, generator=gen)[:topk].to(torch.int32)
            pick[torch.rand(len(pick), generator=gen) < hole] = -1
            ids[b, s, : len(pick)] = pick
    return ids


def check_attention(q, cache, table, cpu, bs, ids, ctx_len, q_start, phase="auto", lse=True, mass=True,
                    p_bits=11, **kw):
    """Runs sparse_attn_q8 and holds out, lse and mass to the reference."""
    dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in kw.items()}
    bt = lci.create_block_table(table.cuda(), cache.k)
    got = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx_len.cuda(), q_start.cuda(), phase=phase,
                             lse=lse, mass=mass, **dev)
    torch.cuda.synchronize()
    lci.get_device_status()
    got = list(got) if isinstance(got, tuple) else [got]
    k, v, ks, vs = cpu
    ro, rl, rm, sizes = ref.attend(q, k.float(), v.float(), ks, vs, table, bs, ids, ctx_len, q_start, **kw)
    hd = q.shape[-1]
    out = got.pop(0).cpu().double()
    assert torch.isfinite(out).all()
    off = (out - ro).abs() / ref.out_tolerance(ro, sizes, q.dtype, hd, 24 if q.dtype == torch.float32 else p_bits)
    assert off.max() <= 1, f"out: {off.max():.2f} of its tolerance at {(off == off.max()).nonzero()[0].tolist()}"
    if lse:
        x = got.pop(0).cpu().double()
        assert torch.equal(x == -float("inf"), rl == -float("inf"))
        fin = rl > -float("inf")
        off = ((x - rl).abs() / ref.lse_tolerance(rl, sizes, hd))[fin]
        assert not fin.any() or off.max() <= 1, f"lse: {off.max():.2f} of its tolerance"
    if mass:
        x = got.pop(0).cpu().double()
        off = (x - rm).abs() / ref.mass_tolerance(rm, sizes, hd, q.shape[2] // cache.k.shape[1])
        assert off.max() <= 1, f"mass: {off.max():.2f} of its tolerance"
    return out


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype,H,bs,hd", [(torch.bfloat16, 1, 64, 128), (torch.float32, 3, 16, 64),
                                           (torch.bfloat16, 2, 48, 40), (torch.float32, 2, 7, 33),
                                           (torch.bfloat16, 1, 128, 256)])
def test_append_matches_the_reference_code_for_code(dtype, H, bs, hd):
    g = torch.Generator().manual_seed(3)
    B, NB = 3, 7
    P = B * NB + 2
    table = make_table(B, NB, P, g)
    cache = make_cache(P, H, bs, hd, g)
    bt = lci.create_block_table(table.cuda(), cache.k)
    state = [vals(cache.k), vals(cache.v), cache.k_scale.cpu().double(), cache.v_scale.cpu().double()]
    at = [0, 5, bs - 1]
    cap = NB * bs
    # a chunk over several blocks, single tokens, a ragged chunk, a chunk inside a block
    for T, ragged, grow in ((2 * bs + 3, False, 1.0), (1, False, 4.0), (1, False, 0.01), (bs + 5, True, 30.0), (3, True, 1.0)):
        k_new = (torch.randn(B, T, H, hd, generator=g) * grow).to(dtype)
        v_new = (torch.randn(B, T, H, hd, generator=g) * grow * 3).to(dtype)
        start = torch.tensor(at, dtype=torch.int32)
        count = torch.tensor([T, 0, T - 1], dtype=torch.int32) if ragged else None
        lci.kv_append_q8(cache, bt, k_new.cuda(), v_new.cuda(), start.cuda(),
                         count=None if count is None else count.cuda())
        torch.cuda.synchronize()
        lci.get_device_status()
        state = ref.append(*state, table, bs, k_new, v_new, start, count)
        for got, want in zip((vals(cache.k), vals(cache.v), cache.k_scale.cpu().double(), cache.v_scale.cpu().double()), state):
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(), want.nan_to_num())
        at = [p + (T if count is None else int(count[b])) for b, p in enumerate(at)]
    assert max(at) <= cap


def test_append_takes_zeros_extremes_infinities_and_nan():
    B, H, bs, hd = 1, 1, 16, 32
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    cache = make_cache(2, H, bs, hd, None)
    bt = lci.create_block_table(table.cuda(), cache.k)
    x = torch.zeros(1, 20, H, hd)
    x[0, 1, 0, 0], x[0, 1, 0, 1] = float("inf"), -float("inf")
    x[0, 2, 0, 5] = float("nan")
    x[0, 3, 0, 7] = 3.0e38
    x[0, 4, 0, 8] = 1e-42
    v = torch.zeros(1, 20, H, hd)
    lci.kv_append_q8(cache, bt, x.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    want = ref.append(torch.full((2, H, bs, hd), float("nan")), torch.full((2, H, bs, hd), float("nan")), torch.ones(2, H), torch.ones(2, H),
                      table, bs, x, v, [0])
    assert torch.equal(vals(cache.k).nan_to_num(nan=-1.0), want[0].nan_to_num(nan=-1.0))
    assert torch.equal(cache.k_scale.cpu().double(), want[2])
    assert float(cache.k_scale[1, 0]) == 2.0 ** 120 and float(cache.v_scale[1, 0]) == 2.0 ** -60
    k = vals(cache.k)
    assert k[1, 0, 1, 0] == 448 and k[1, 0, 1, 1] == -448 and k[1, 0, 2, 5].isnan()


def test_append_to_scales_from_elsewhere():
    """Stored scales that are no powers of two stay where they are large enough."""
    g = torch.Generator().manual_seed(9)
    bs, hd = 16, 64
    table = torch.tensor([[0]], dtype=torch.int32)
    cache = lci.Q8Cache(1, 1, bs, hd, "cuda")
    cache.k.copy_((torch.randn(1, 1, bs, hd, generator=g) * 100).clamp(-448, 448).to(E4M3))
    cache.k_scale.fill_(0.3)
    state = [vals(cache.k), vals(cache.v), cache.k_scale.cpu().double(), cache.v_scale.cpu().double()]
    bt = lci.create_block_table(table.cuda(), cache.k)
    for p, mult in ((4, 1.0), (5, 1000.0)):
        new = torch.randn(1, 1, 1, hd, generator=g) * mult
        lci.kv_append_q8(cache, bt, new.cuda(), new.cuda(), torch.tensor([p], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        s = float(cache.k_scale[0, 0])
        old = state[2][0, 0].item()
        assert s == max(old, ref.needed_scale(float(new.abs().max())))
        # one fp32 division, then one rounding
        want = (new.float() / cache.k_scale.cpu()[0, 0]).to(E4M3).float().double()
        assert torch.equal(vals(cache.k)[0, 0, p], want[0, 0, 0])
        state[2][0, 0] = s


def test_append_flags_what_it_skips():
    cache = make_cache(4, 1, 16, 32, None)
    bt = lci.create_block_table(torch.tensor([[0, 9], [2, 3]], dtype=torch.int32, device="cuda"), cache.k)
    new = torch.ones(2, 1, 1, 32, device="cuda")
    for start in ([16, 0], [40, 0], [-1, 0]):  # a bad page, a block past the table, a negative start
        before = cache.k.view(torch.uint8).clone()
        lci.kv_append_q8(cache, bt, new, new, torch.tensor(start, dtype=torch.int32, device="cuda"))
        with pytest.raises(lci.LciError) as e:
            lci.get_device_status()
        assert e.value.status == 5
        after = cache.k.view(torch.uint8)
        changed = (before != after).nonzero()
        assert (changed[:, 0] == 2).all()  # only the good sequence's page


# ---------------------------------------------------------------- attention

SHAPES = [  # dtype, B, S, ctx, H_kv, G, hd, bs, topk
    (torch.bfloat16, 2, 1, 300, 1, 16, 128, 64, 4),
    (torch.bfloat16, 1, 1, 1, 1, 1, 128, 64, 1),
    (torch.bfloat16, 3, 2, 500, 2, 8, 128, 64, 9),
    (torch.bfloat16, 1, 3, 900, 1, 5, 128, 128, 7),
    (torch.bfloat16, 1, 37, 700, 2, 4, 128, 64, 6),
    (torch.bfloat16, 1, 70, 1100, 1, 16, 128, 64, 8),
    (torch.bfloat16, 2, 33, 520, 1, 8, 128, 128, 3),
    (torch.bfloat16, 1, 2, 300, 1, 16, 64, 64, 3),
    (torch.bfloat16, 1, 2, 90, 2, 3, 128, 16, 4),
    (torch.bfloat16, 1, 2, 200, 1, 20, 128, 64, 3),
    (torch.float32, 2, 5, 100, 2, 2, 64, 16, 4),
    (torch.float32, 1, 3, 77, 1, 1, 32, 8, 5),
    (torch.float32, 1, 2, 200, 1, 3, 256, 48, 5),
    (torch.float32, 1, 2, 300, 1, 4, 128, 64, 5),
]


def attention_inputs(shape, seed, spread=2.0):
    dtype, B, S, ctx, H, G, hd, bs, topk = shape
    g = torch.Generator().manual_seed(seed)
    lens = [max(S if ctx >= S else 1, ctx - 29 * b) for b in range(B)]
    cache, table, cpu = filled_cache(B, H, bs, hd, lens, seed + 1, spread)
    q = torch.randn(B, S, H * G, hd, generator=g).to(dtype)
    ctx_len = torch.tensor(lens, dtype=torch.int32)
    ids = random_ids(B, S, table.shape[1], topk, g)
    return q, cache, table, cpu, bs, ids, ctx_len, ctx_len - S


@pytest.mark.parametrize("phase", ["auto", "prefill", "decode"])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_matches_the_reference(shape, phase):
    check_attention(*attention_inputs(shape, 20), phase=phase, mass=phase != "prefill",
                    p_bits=8 if phase != "decode" else 11)


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("mods", ["cap", "slopes", "docs", "prefix", "all"])
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2], SHAPES[3], SHAPES[4], SHAPES[5], SHAPES[8], SHAPES[10]])
def test_changed_scores_match_the_reference(shape, mods, phase):
    args = attention_inputs(shape, 30)
    q, ctx_len, q_start = args[0], args[6], args[7]
    B, S, Hq, _ = q.shape
    p = q_start[:, None] + torch.arange(S, dtype=torch.int32)[None]
    kw = {}
    if mods in ("cap", "all"):
        kw["cap"] = 3.0
    if mods in ("slopes", "all"):
        kw["slopes"] = torch.exp2(-8.0 * (torch.arange(Hq) + 1) / Hq).float()
    if mods in ("docs", "all"):
        kw["first"] = ((p // 45) * 45).to(torch.int32).contiguous()
    if mods in ("prefix", "all"):
        kw["last"] = p.clamp(min=150).to(torch.int32).contiguous()
    check_attention(*args, phase=phase, mass=phase != "prefill", p_bits=8 if phase == "prefill" else 11, **kw)


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[5], SHAPES[10]])
def test_rows_without_a_token_are_zero(shape, phase):
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(shape, 40)
    B, S = q.shape[:2]
    p = q_start[:, None] + torch.arange(S, dtype=torch.int32)[None]
    ids[0, 0] = -1                                   # nothing selected
    ctx_len[-1] = 0                                  # an empty sequence
    first = torch.zeros_like(p)
    first[0, S - 1] = int(p[0, S - 1]) + 1            # a window behind the query
    out = check_attention(q, cache, table, cpu, bs, ids, ctx_len, q_start, phase=phase, mass=phase != "prefill",
                          p_bits=8 if phase == "prefill" else 11, first=first.contiguous())
    assert (out[0, 0] == 0).all() and (out[-1] == 0).all() and (out[0, S - 1] == 0).all()


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("case", ["wide_scales", "large_scores", "one_token", "tiny_v", "zero_v"])
def test_scales_and_scores_far_apart(case, phase):
    shape = SHAPES[5]
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(shape, 50)
    k, v, ks, vs = cpu
    if case == "wide_scales":
        g = torch.Generator().manual_seed(1)
        vs.mul_(torch.exp2(torch.randint(-20, 20, vs.shape, generator=g).float()))
    if case == "large_scores":
        q.mul_(40)
    if case == "one_token":
        ids[:, :, 1:] = -1
        ids[:, :, 0] = 0
        ctx_len[:] = 1
    if case == "tiny_v":
        vs.mul_(2.0 ** -50)
    if case == "zero_v":
        v.copy_(torch.zeros_like(v.float()).to(E4M3))
        vs.fill_(2.0 ** -60)
    cache = lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs)))
    check_attention(q, cache, table, (k, v, ks, vs), bs, ids, ctx_len, q_start, phase=phase, mass=phase != "prefill",
                    p_bits=8 if phase == "prefill" else 11)


@pytest.mark.parametrize("phase", ["prefill", "decode"])
def test_nan_reaches_only_the_rows_that_attend_it(phase):
    """A NaN inside the context: rows that attend it are NaN in its channel, rows
    that mask it or did not select its block are what they are without it."""
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(SHAPES[5], 60)
    k, v, ks, vs = cpu
    t_bad = int(ctx_len[0]) - 40  # some queries are before it, some after
    page = int(table[0, t_bad // bs])
    clean = v.clone()
    v.view(torch.uint8)[page, 0, t_bad % bs, 17] = 0x7F
    cache = lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs)))
    bt = lci.create_block_table(table.cuda(), cache.k)
    out = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx_len.cuda(), q_start.cuda(), phase=phase).cpu().double()
    lci.get_device_status()
    ro, _, _, sizes = ref.attend(q, k.float(), clean.float(), ks, vs, table, bs, ids, ctx_len, q_start)
    S = q.shape[1]
    hit = torch.tensor([t_bad // bs in ids[0, s].tolist() and int(q_start[0]) + s >= t_bad for s in range(S)])
    assert hit.any() and not hit.all()
    assert out[0, hit][:, :, 17].isnan().all()
    keep = torch.arange(128) != 17
    assert torch.isfinite(out[0, hit][:, :, keep]).all() and torch.isfinite(out[0, ~hit]).all()
    off = (out - ro).abs() / ref.out_tolerance(ro, sizes, q.dtype, 128, 8)
    assert off[0, ~hit].max() <= 1 and off[0, hit][:, :, keep].max() <= 1


def test_bad_ids_and_pages_are_skipped_and_flagged():
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(SHAPES[0], 70)
    ids[:, :, 0] = torch.tensor([0, 1], dtype=torch.int32)[:, None]
    for phase in ("prefill", "decode"):
        for what in ("id", "page"):
            t2, i2 = table.clone(), ids.clone()
            if what == "id":
                i2[0, 0, 1] = table.shape[1] + 3
            else:
                i2[0, 0, :2] = torch.tensor([0, 2], dtype=torch.int32)
                t2[0, 2] = 10 ** 6
            bt = lci.create_block_table(t2.cuda(), cache.k)
            lci.sparse_attn_q8(q.cuda(), cache, bt, i2.cuda(), ctx_len.cuda(), q_start.cuda(), phase=phase)
            with pytest.raises(lci.LciError) as e:
                lci.get_device_status()
            assert e.value.status == 5


def test_other_streams_and_captured_calls_give_the_same():
    args = attention_inputs(SHAPES[2], 80)
    q, cache, table, cpu, bs, ids, ctx_len, q_start = args
    bt = lci.create_block_table(table.cuda(), cache.k)
    dev = [t.cuda() for t in (q, ids, ctx_len, q_start)]
    call = lci.prepare_sparse_attn_q8(dev[0], cache, bt, dev[1], dev[2], dev[3], lse=True, mass=True)
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in call.result:
        t.fill_(-5)
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(call.result, want))
    for t in call.result:
        t.fill_(-5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(call.result, want))
    lci.get_device_status()


WIDE = [  # tiles of many blocks, odd head groups, several KV heads, lists longer than what is visible
    (torch.bfloat16, 1, 40, 38500, 1, 4, 128, 64, 64),
    (torch.bfloat16, 1, 45, 900, 4, 3, 128, 64, 200),
    (torch.bfloat16, 2, 19, 400, 1, 7, 128, 128, 5),
    (torch.bfloat16, 1, 33, 330, 2, 1, 128, 64, 4),
    (torch.bfloat16, 1, 9, 1030, 1, 13, 128, 192, 6),
    (torch.bfloat16, 90, 4, 250, 1, 2, 128, 64, 5),
    (torch.bfloat16, 40, 4, 250, 2, 8, 64, 16, 20),
]


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("shape", WIDE)
def test_wide_unions_and_odd_groups(shape, phase):
    check_attention(*attention_inputs(shape, 90), phase=phase, mass=phase != "prefill", p_bits=8 if phase == "prefill" else 11)


def test_cells_past_four_gigabytes():
    """Pools of 4.5 GB: the last pages' bytes lie past 32-bit offsets."""
    H, bs, hd, P, n = 1, 128, 128, 275000, 300
    cache = lci.Q8Cache(P, H, bs, hd, "cuda")
    table = torch.tensor([[P - 1, 3, P - 2], [P - 3, P - 4, 5]], dtype=torch.int32)
    bt = lci.create_block_table(table.cuda(), cache.k)
    g = torch.Generator().manual_seed(2)
    k_new, v_new = (torch.randn(2, n, H, hd, generator=g).to(torch.bfloat16) for _ in range(2))
    start = torch.zeros(2, dtype=torch.int32)
    lci.kv_append_q8(cache, bt, k_new.cuda(), v_new.cuda(), start.cuda())
    pages = table.flatten().long()
    small = [t[pages.cuda()].cpu() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
    local = torch.arange(6, dtype=torch.int32).reshape(2, 3)
    want = ref.append(torch.zeros(6, H, bs, hd), torch.zeros(6, H, bs, hd), torch.ones(6, H), torch.ones(6, H), local, bs, k_new, v_new, start)
    assert torch.equal(small[0].view(E4M3).float().double(), want[0]) and torch.equal(small[3].double(), want[3])
    S = 24
    q = torch.randn(2, S, 16, hd, generator=g).to(torch.bfloat16)
    ids = random_ids(2, S, 3, 3, g, hole=0.0)
    ctx = torch.tensor([n, n], dtype=torch.int32)
    ro, _, _, sizes = ref.attend(q, want[0], want[1], want[2], want[3], local, bs, ids, ctx, ctx - S)
    for phase, bits in (("prefill", 8), ("decode", 11)):
        out = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx.cuda(), (ctx - S).cuda(), phase=phase)
        torch.cuda.synchronize()
        lci.get_device_status()
        assert ((out.cpu().double() - ro).abs() <= ref.out_tolerance(ro, sizes, q.dtype, hd, bits)).all()


def test_calls_on_two_streams_at_once():
    """Two caches, two tables, two streams, no shared state: each call's result is
    what it is alone."""
    made = []
    for i, shape in enumerate((SHAPES[5], SHAPES[4], SHAPES[0])):
        q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(shape, 100 + i)
        bt = lci.create_block_table(table.cuda(), cache.k)
        call = lci.prepare_sparse_attn_q8(*(x.cuda() if isinstance(x, torch.Tensor) else x for x in (q, cache, bt, ids, ctx_len, q_start)), lse=True)
        made.append((call, [t.clone() for t in call()]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(20):
        for st, (call, _) in zip(streams, made):
            call(st)
    torch.cuda.synchronize()
    lci.get_device_status()
    for call, want in made:
        assert all(torch.equal(a, b) for a, b in zip(call.result, want))


def test_refusals_of_the_binding():
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(SHAPES[0], 110)
    bt = lci.create_block_table(table.cuda(), cache.k)
    d = [t.cuda() for t in (q, ids, ctx_len, q_start)]
    with pytest.raises(ValueError):  # not contiguous
        lci.sparse_attn_q8(d[0].transpose(1, 2).contiguous().transpose(1, 2)[:, :, ::2], cache, bt, d[1], d[2], d[3])
    with pytest.raises(TypeError):
        lci.sparse_attn_q8(d[0].half(), cache, bt, d[1], d[2], d[3])
    with pytest.raises(ValueError):
        lci.sparse_attn_q8(d[0], cache, bt, d[1], d[2][:1], d[3])
    with pytest.raises(ValueError):
        lci.sparse_attn_q8(d[0], cache, bt, d[1], d[2], d[3], slopes=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        lci.sparse_attn_q8(d[0], cache, bt, d[1], d[2], d[3], first=torch.zeros(2, 1, device="cuda"))
    with pytest.raises(ValueError):
        lci.sparse_attn_q8(d[0], cache, bt, d[1], d[2], d[3].cpu())
    with pytest.raises(ValueError):  # another cache's pools
        lci.sparse_attn_q8(d[0], lci.Q8Cache(3, 1, 64, 128, "cuda"), bt, d[1], d[2], d[3])
    with pytest.raises(TypeError):  # a table over bf16 pools
        lci.kv_append_q8(cache, lci.create_block_table(table.cuda(), cache.k.to(torch.bfloat16)), torch.zeros(2, 1, 1, 128, device="cuda"),
                         torch.zeros(2, 1, 1, 128, device="cuda"), d[2])
    with pytest.raises(lci.LciError):
        lci.cache_evict(bt, d[2], torch.zeros(table.shape, device="cuda"), 3, sink=2, recent=2)
    with pytest.raises(lci.LciError):
        lci.block_weight_update(torch.zeros(2, 5, device="cuda"), d[1], torch.zeros(2, 1, 1, 4, device="cuda"), decay=-1.0)
    with pytest.raises(lci.LciError):  # the bf16 attention does not take this table
        lci.sparse_attn_workspace_size(2, 1, 16, 4, bt)


@pytest.mark.parametrize("dtype,H,G,hd,bs,topk", [(torch.float32, 2, 11, 64, 16, 5), (torch.float32, 1, 8, 96, 48, 3),
                                                  (torch.bfloat16, 2, 17, 128, 64, 4), (torch.float32, 1, 40, 32, 8, 256),
                                                  (torch.bfloat16, 1, 3, 256, 24, 7)])
@pytest.mark.parametrize("mass", [False, True])
def test_cuda_core_schedule_with_many_heads(dtype, H, G, hd, bs, topk, mass):
    """The heads of a KV head over CTAs, their masses added up across them."""
    lens = [topk * bs + 3, bs - 1]
    B, S = 2, 3
    cache, table, cpu = filled_cache(B, H, bs, hd, lens, 31)
    g = torch.Generator().manual_seed(32)
    NB = table.shape[1]
    ids = random_ids(B, S, NB, topk, g)
    q = torch.randn(B, S, H * G, hd, generator=g).to(dtype)
    ctx = torch.tensor(lens, dtype=torch.int32)
    check_attention(q, cache, table, cpu, bs, ids, ctx, (ctx - S).clamp(min=0).to(torch.int32), mass=mass,
                    cap=20.0, slopes=torch.rand(H * G, generator=g) / 8)


# ---------------------------------------------------------------- weights and eviction

@pytest.mark.parametrize("B,S,H,topk,NB,decay", [(1, 1, 1, 1, 1, 1.0), (3, 1, 2, 8, 40, 0.5), (2, 70, 1, 32, 100, 1.0),
                                                 (1, 700, 2, 5, 1025, 0.9), (2, 9, 1, 256, 2500, 0.0), (1, 2100, 1, 3, 16384, 1.0)])
def test_block_weights_accumulate(B, S, H, topk, NB, decay):
    g = torch.Generator().manual_seed(5)
    ids = random_ids(B, S, NB, topk, g)
    mass = torch.rand(B, S, H, topk, generator=g) ** 6
    weight = torch.rand(B, NB, generator=g)
    got = lci.block_weight_update(weight.cuda(), ids.cuda(), mass.cuda(), decay=decay)
    again = lci.block_weight_update(weight.cuda(), ids.cuda(), mass.cuda(), decay=decay)
    torch.cuda.synchronize()
    lci.get_device_status()
    want = ref.weight_update(weight, ids, mass, decay)
    # fp32 sums of at most S addends in each warp, one rounding of the total
    tol = want * 2.0 ** -24 * (H + 2 + S) + 1e-30
    assert ((got.cpu().double() - want).abs() <= tol).all()
    assert torch.equal(got, again)


@pytest.mark.parametrize("B,S,H,topk,NB", [(1, 4, 8, 32, 1024), (2, 2, 3, 33, 1025), (1, 38, 2, 97, 104), (3, 73, 4, 256, 300),
                                           (2, 300, 8, 64, 2048), (1, 1100, 2, 200, 1200)])
def test_block_weights_of_wide_rows_and_many_heads(B, S, H, topk, NB):
    """Rows of several runs of 32 entries, masses of many heads, and -1 entries whose masses do not count."""
    g = torch.Generator().manual_seed(7)
    ids = random_ids(B, S, NB, topk, g)
    ids[torch.rand(ids.shape, generator=g) < 0.2] = -1
    mass = torch.rand(B, S, H, topk, generator=g) ** 6
    mass[(ids < 0)[:, :, None, :].expand_as(mass)] = float("nan")
    weight = torch.rand(B, NB, generator=g)
    got = lci.block_weight_update(weight.cuda(), ids.cuda(), mass.cuda(), decay=0.5)
    again = lci.block_weight_update(weight.cuda(), ids.cuda(), mass.cuda(), decay=0.5)
    torch.cuda.synchronize()
    lci.get_device_status()
    mass[mass != mass] = 0.0
    want = ref.weight_update(weight, ids, mass, 0.5)
    tol = want * 2.0 ** -24 * (H + 2 + S) + 1e-30
    assert ((got.cpu().double() - want).abs() <= tol).all()
    assert torch.equal(got, again)


def test_block_weights_flag_bad_ids():
    ids = torch.tensor([[[0, 7, -1, -3]]], dtype=torch.int32, device="cuda")
    w = lci.block_weight_update(torch.zeros(1, 4, device="cuda"), ids, torch.ones(1, 1, 1, 4, device="cuda"))
    with pytest.raises(lci.LciError):
        lci.get_device_status()
    assert w.tolist() == [[1.0, 0.0, 0.0, 0.0]]


@pytest.mark.parametrize("B,NB,bs,budget,sink,recent,levels", [
    (1, 1, 64, 1, 0, 1, 0), (3, 40, 16, 17, 1, 3, 0), (2, 512, 64, 100, 4, 8, 3), (2, 1500, 64, 700, 0, 1, 0),
    (1, 5000, 64, 4999, 2, 3, 2), (1, 16384, 64, 300, 7, 29, 0), (4, 33, 64, 40, 1, 1, 0), (2, 100, 64, 5, 2, 3, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_matches_the_reference(B, NB, bs, budget, sink, recent, levels, in_place):
    g = torch.Generator().manual_seed(7)
    table = make_table(B, NB, B * NB + 1, g)
    ctx = torch.tensor([max(0, NB * bs - 3 - b * (NB * bs // 4)) for b in range(B)], dtype=torch.int32)
    weight = torch.randn(B, NB, generator=g) ** 3
    if levels:
        weight = torch.randint(0, levels, (B, NB), generator=g).float()
    want = ref.evict(table, ctx, weight, bs, budget, sink, recent)
    bt = lci.BlockTable(table.cuda(), B * NB + 1, bs, 1, 128, E4M3)
    d_ctx, d_w = ctx.cuda(), weight.cuda()
    got = lci.cache_evict(bt, d_ctx, d_w, budget, sink=sink, recent=recent, in_place=in_place)
    torch.cuda.synchronize()
    lci.get_device_status()
    for name, a, b in zip(("table", "ctx_len", "weight", "kept", "freed"), got, want):
        assert torch.equal(a.cpu(), b), name
    assert (got[0].data_ptr() == bt.table.data_ptr()) == in_place
    if not in_place:
        assert torch.equal(bt.table.cpu(), table) and torch.equal(d_ctx.cpu(), ctx) and torch.equal(d_w.cpu(), weight)


def test_eviction_of_special_weights_and_lengths():
    nan, inf = float("nan"), float("inf")
    weight = torch.tensor([[0.0, -0.0, nan, inf, -inf, 0.0, 5.0, 1.0], [1, 2, 3, 4, 5, 6, 7, 8], [1, 2, 3, 4, 5, 6, 7, 8],
                           [1, 2, 3, 4, 5, 6, 7, 8]])
    table = torch.arange(32, dtype=torch.int32).reshape(4, 8)
    ctx = torch.tensor([128, 0, 16, 8 * 16 + 1], dtype=torch.int32)  # full, empty, one block, longer than its row
    bt = lci.BlockTable(table.cuda(), 32, 16, 1, 128, torch.bfloat16)
    t, c, w, kept, freed = lci.cache_evict(bt, ctx.cuda(), weight.cuda(), 5, sink=0, recent=1, in_place=False)
    with pytest.raises(lci.LciError):
        lci.get_device_status()
    # kept: the last, NaN, inf, 5, and of the zeros the lowest block
    assert kept[0].tolist() == [0, 2, 3, 6, 7] and freed.tolist() == [3, 0, 0, 0]
    assert t[0].tolist() == [0, 2, 3, 6, 7, 1, 4, 5] and c.tolist() == [80, 0, 16, 129]
    assert t[3].tolist() == table[3].tolist() and w[3].tolist() == weight[3].tolist()
    assert kept[1].tolist() == [-1] * 5 and kept[2].tolist() == [0, -1, -1, -1, -1]


def test_captured_serving_step_replays():
    """Append, attention with masses and the weights' update as one graph, replayed
    with new inputs in the same buffers, against the same calls made one by one."""
    B, H, G, hd, bs, NB = 3, 2, 4, 128, 64, 5
    g = torch.Generator().manual_seed(13)
    table = make_table(B, NB, B * NB, g).cuda()
    state = []
    for _ in range(2):
        cache = lci.Q8Cache(B * NB, H, bs, hd, "cuda")
        state.append((cache, lci.create_block_table(table, cache.k), torch.zeros(B, NB, device="cuda")))
    new = [torch.zeros(B, 1, H, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = torch.zeros(B, 1, H * G, hd, dtype=torch.bfloat16, device="cuda")
    pos = torch.full((B,), 70, dtype=torch.int32, device="cuda")
    ctx = pos + 1
    ids = torch.tensor([1, 0, -1], dtype=torch.int32, device="cuda").repeat(B, 1, 1)

    def step(cache, bt, weight):
        lci.kv_append_q8(cache, bt, new[0], new[1], pos)
        out, mass = lci.sparse_attn_q8(q, cache, bt, ids, ctx, pos, mass=True)
        lci.block_weight_update(weight, ids, mass, decay=0.5)
        return out
    prompt = [torch.randn(B, 70, H, hd, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    for cache, bt, _ in state:
        lci.kv_append_q8(cache, bt, prompt[0], prompt[1], torch.zeros_like(pos))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out_g = step(*state[0])
    for t in range(4):
        for x in new + [q]:
            x.copy_(torch.randn(x.shape, generator=g) * (1 + t))
        pos.fill_(70 + t)
        ctx.copy_(pos + 1)
        graph.replay()
        out = step(*state[1])
        torch.cuda.synchronize()
        assert torch.equal(out, out_g) and torch.equal(state[0][2], state[1][2])
        assert torch.equal(state[0][0].k.view(torch.uint8), state[1][0].k.view(torch.uint8))
    lci.get_device_status()


# ---------------------------------------------------------------- together

def test_a_bounded_decode_loop():
    """Prompt, then decode steps: append, block keys, selection through the
    table, attention with the blocks' weights, their accumulation, eviction.
    Every step is held to the reference on the cache's own state."""
    g = torch.Generator().manual_seed(11)
    B, H, G, hd, bs, topk, NB, budget = 2, 1, 16, 128, 64, 4, 10, 6
    P = B * NB
    table = make_table(B, NB, P, g).cuda()
    cache = lci.Q8Cache(P, H, bs, hd, "cuda")
    bt = lci.create_block_table(table, cache.k)
    keys = lci.PagedKeys(P, 1, 64, torch.bfloat16, "cuda")
    weight = torch.zeros(B, NB, device="cuda")
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    evicted = 0
    for step, T in enumerate([bs * 5 + 20, 1, 1, 43, 1, 64, 1, 1, 64, 1]):
        k_new, v_new = (torch.randn(B, T, H, hd, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        k_idx = (torch.randint(-32, 33, (B, T, 1, 64), generator=g) / 16).to(torch.bfloat16).cuda()
        q = torch.randn(B, T, H * G, hd, generator=g).to(torch.bfloat16).cuda()
        q_c = (torch.randint(-32, 33, (B, T, 1, 64), generator=g) / 16).to(torch.bfloat16).cuda()
        start = ctx.clone()
        cache.append(k_new, v_new, start, bt)
        keys.update(k_idx, start, bt)
        ctx += T
        ids = lci.index_select_paged(q_c, keys, bt, ctx, start, topk)
        out, mass = lci.sparse_attn_q8(q, cache, bt, ids, ctx, start, mass=True)
        lci.block_weight_update(weight, ids, mass, decay=0.9)
        torch.cuda.synchronize()
        lci.get_device_status()
        rows = slice(max(0, T - 3), T)  # the reference on the last queries
        ro, _, rm, sizes = ref.attend(q.cpu()[:, rows], cache.k.cpu().float(), cache.v.cpu().float(), cache.k_scale.cpu(), cache.v_scale.cpu(),
                                      table.cpu(), bs, ids.cpu()[:, rows], ctx.cpu(), start.cpu() + max(0, T - 3))
        assert ((out.cpu().double()[:, rows] - ro).abs() <= ref.out_tolerance(ro, sizes, q.dtype, hd, 8)).all()
        assert ((mass.cpu().double()[:, rows] - rm).abs() <= ref.mass_tolerance(rm, sizes, hd, G)).all()
        before = [t.cpu().clone() for t in (table, ctx, weight)]
        _, _, _, _, freed = lci.cache_evict(bt, ctx, weight, budget, sink=1, recent=2)
        want = ref.evict(*before, bs, budget, 1, 2)
        assert torch.equal(table.cpu(), want[0]) and torch.equal(ctx.cpu(), want[1]) and torch.equal(weight.cpu(), want[2])
        evicted += int(freed.sum())
    assert evicted > 0 and sorted(table.flatten().tolist()) == list(range(P))


def test_tiles_whose_queries_share_no_block():
    """Every query picks blocks of its own, so that most of a tile's warps only
    pass the softmax references on: many rounds of the same call give the same."""
    g = torch.Generator().manual_seed(120)
    B, S, G, bs, hd, topk = 1, 48, 16, 64, 128, 6
    NB = S * topk
    cache, table, cpu = filled_cache(B, 1, bs, hd, [NB * bs], 121)
    q = torch.randn(B, S, G, hd, generator=g).to(torch.bfloat16)
    ids = torch.randperm(NB, generator=g).reshape(1, S, topk).to(torch.int32)
    ctx = torch.tensor([NB * bs], dtype=torch.int32)
    args = (q, cache, table, cpu, bs, ids, ctx, ctx - S)
    first = check_attention(*args, phase="prefill", mass=False, p_bits=8)
    bt = lci.create_block_table(table.cuda(), cache.k)
    call = lci.prepare_sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx.cuda(), (ctx - S).cuda(), phase="prefill")
    for _ in range(50):
        call()
    torch.cuda.synchronize()
    lci.get_device_status()
    assert torch.equal(call.result.cpu().double(), first)


def test_tiles_that_give_up_leave_zeros():
    """With a limit that nearly every wait exceeds, tiles give up: each of their rows
    is zero, or what it should be where the tile got through, and never raw codes."""
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(SHAPES[5], 130)
    bt = lci.create_block_table(table.cuda(), cache.k)
    dev = [t.cuda() for t in (q, ids, ctx_len, q_start)]
    call = lci.prepare_sparse_attn_q8(dev[0], cache, bt, *dev[1:], phase="prefill", lse=True)
    want = [t.clone() for t in call()]
    default = lci.get_wait_limit_ns()
    lci.set_wait_limit_ns(1)
    try:
        for _ in range(5):
            for t in call.result:
                t.fill_(7.0)
            call()
            try:
                lci.get_device_status()
                timed_out = False
            except lci.LciError as e:
                assert e.status == 6
                timed_out = True
            zero = (call.result[0] == 0).all(-1) & (call.result[1] == -float("inf"))
            same = (call.result[0] == want[0]).all(-1) & (call.result[1] == want[1])
            assert (zero | same).all() and (timed_out or same.all())
    finally:
        lci.set_wait_limit_ns(default)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    lci.get_device_status()


def check_shares(q, k, v, ks, vs, table, bs, ids, ctx, phase):
    """Output of each channel against what the channel's own tokens add up to."""
    cache = lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs)))
    bt = lci.create_block_table(table.cuda(), cache.k)
    S, hd = q.shape[1], q.shape[3]
    out = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx.cuda(), (ctx - S).cuda(), phase=phase)
    torch.cuda.synchronize()
    lci.get_device_status()
    ro, _, _, sizes = ref.attend(q, k.float(), v.float(), ks, vs, table, bs, ids, ctx, ctx - S)
    share = ref.attend(q, k.float(), v.float().abs(), ks, vs, table, bs, ids, ctx, ctx - S)[0]
    floor = ref.weight_floor(q, k.float(), v.float(), ks, vs, table, bs, ids, ctx, ctx - S)
    off = (out.cpu().double() - ro).abs()
    assert (off <= ref.out_tolerance(ro, sizes, q.dtype, hd, 8 if phase == "prefill" else 11)).all()
    off = off / ref.share_tolerance(ro, share, floor, sizes, q.dtype, hd, 8 if phase == "prefill" else 11)
    assert off.max() <= 1, f"{off.max():.2f} of its tolerance"


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("sink", [0.5, 0.7, 0.9, 0.99])
@pytest.mark.parametrize("nblk,bs", [(32, 64), (128, 64), (256, 64), (256, 128)])
def test_a_sink_leaves_the_other_tokens_their_share(nblk, bs, sink, phase):
    """One token takes most of the softmax and has no value: the many small
    weights behind it are the whole output."""
    g = torch.Generator().manual_seed(140)
    S, G, hd, n = 2, 4, 128, nblk * bs
    q = torch.randn(1, S, G, hd, generator=g)
    q[..., 0] = 8.0
    q = q.to(torch.bfloat16)
    k = torch.randn(nblk, 1, bs, hd, generator=g) * 0.5   # scores of about half a nat
    v = torch.randn(nblk, 1, bs, hd, generator=g) * 0.5 + 0.5
    k[..., 0] = 0.0
    table = torch.randperm(nblk, generator=g).to(torch.int32)[None].contiguous()
    page = int(table[0, 0])
    k[page, 0, 0], v[page, 0, 0] = 0.0, 0.0
    k[page, 0, 0, 0] = (math.log(sink / (1 - sink) * n) + 0.125) * math.sqrt(hd) / 8.0
    ks = torch.full((nblk, 1), 2.0 ** -4)
    vs = torch.full((nblk, 1), 2.0 ** -6)
    k, v = ((x / s[:, :, None, None]).clamp(-448, 448).to(E4M3) for x, s in ((k, ks), (v, vs)))
    ids = torch.stack([torch.randperm(nblk, generator=g) for _ in range(S)])[None].to(torch.int32)
    check_shares(q, k, v, ks, vs, table, bs, ids, torch.tensor([n], dtype=torch.int32), phase)


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("apart", [8, 12, 14, 17, 20])
def test_pages_whose_v_scales_are_far_apart(apart, phase):
    """Every fourth page's v scale is 2^apart of the others', and its values are in
    channels of their own: the other channels are the small pages' alone."""
    g = torch.Generator().manual_seed(141)
    S, G, hd, bs, nblk = 5, 8, 128, 64, 12
    q = torch.randn(1, S, G, hd, generator=g).to(torch.bfloat16)
    k = torch.randn(nblk, 1, bs, hd, generator=g)
    v = torch.randn(nblk, 1, bs, hd, generator=g) * 100
    table = torch.randperm(nblk, generator=g).to(torch.int32)[None].contiguous()
    big = torch.arange(nblk) % 4 == 1
    v[big, :, :, 64:] = 0.0
    v[~big, :, :, :64] = 0.0
    ks = torch.full((nblk, 1), 2.0 ** -6)
    vs = torch.where(big, 2.0 ** apart, 1.0)[:, None] * 1.25
    k, v = (k * 64).clamp(-448, 448).to(E4M3), v.clamp(-448, 448).to(E4M3)
    ids = torch.stack([torch.randperm(nblk, generator=g) for _ in range(S)])[None].to(torch.int32)
    check_shares(q, k, v, ks, vs, table, bs, ids, torch.tensor([nblk * bs], dtype=torch.int32), phase)


def capped_inputs(seed, S=40, G=8, ctx=700, bs=64, hd=128):
    """Keys along the queries, with codes up to the largest: raw products of 2^19 and more."""
    g = torch.Generator().manual_seed(seed)
    base = torch.randn(hd, generator=g)
    q = (base * (1 + 0.05 * torch.randn(1, S, G, hd, generator=g))).to(torch.bfloat16)
    cache, table, cpu = filled_cache(1, 1, bs, hd, [ctx], seed + 1)
    k, v, ks, vs = cpu
    along = 2 * torch.rand(k.shape[:3], generator=g) - 1
    x = (along[..., None] * base * (1 + 0.05 * torch.randn(k.shape, generator=g)))
    codes = (x / x.abs().max() * 448).clamp(-448, 448).to(E4M3)
    raw = k.view(torch.uint8)
    raw.copy_(torch.where(raw == 0x7F, raw, codes.view(torch.uint8)))  # NaN stays behind the context
    ks.fill_(2.0 ** -7)
    ids = torch.stack([torch.randperm(table.shape[1], generator=g) for _ in range(S)])[None].to(torch.int32)
    ctx_len = torch.tensor([ctx], dtype=torch.int32)
    p = (ctx_len - S)[:, None] + torch.arange(S, dtype=torch.int32)[None]
    # the largest attended product, so that a softmax scale sets the largest |z| / cap
    keys = (k.float().nan_to_num(0.0) * ks[:, :, None, None])[table[0].long()].permute(1, 0, 2, 3).reshape(-1, hd)[:ctx]
    top = float((q.float().reshape(-1, hd) @ keys.T).abs().max())
    return lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs))), q, table, cpu, bs, ids, ctx_len, ctx_len - S, top


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("u", [0.2, 0.4, 0.6, 2.0])
@pytest.mark.parametrize("cap", [20.0, 30.0, 50.0, 1000.0])
def test_caps_over_the_range_of_the_hyperbolic_tangent(cap, u, phase):
    """Scores up to u times the cap, for each way that tanh is computed."""
    cache, q, table, cpu, bs, ids, ctx_len, q_start, top = capped_inputs(150)
    check_attention(q, cache, table, cpu, bs, ids, ctx_len, q_start, phase=phase, mass=phase != "prefill",
                    p_bits=8 if phase == "prefill" else 11, cap=cap, scale=u * cap / top)


@pytest.mark.parametrize("phase", ["prefill", "decode"])
@pytest.mark.parametrize("u", [0.2, 0.55])
def test_slots_that_are_not_attended_change_no_bit(u, phase):
    """What lies behind the context, and tokens outside a query's window: NaN, zero
    and the largest codes of either sign give the same bits, under a cap too."""
    cache, q, table, cpu, bs, ids, ctx_len, q_start, top = capped_inputs(160, S=12, ctx=460)
    S, n, cap = q.shape[1], int(ctx_len[0]), 30.0
    p = int(q_start[0]) + torch.arange(S, dtype=torch.int32)
    first = torch.full((1, S), 70, dtype=torch.int32)   # tokens 0 .. 69 are behind every window
    last = torch.minimum(p, torch.tensor(400)).to(torch.int32)[None]
    bt = lci.create_block_table(table.cuda(), cache.k)
    hide = torch.ones(table.shape[1] * bs, dtype=torch.bool)
    hide[70:401] = False
    seen = []
    along = torch.where(q[0, 0, 0] > 0, 0x7E, 0xFE).to(torch.uint8).cuda()  # +-448 along the queries
    for code in (0x00, 0x7F, along, along ^ 0x80):  # 0, NaN, the largest products of either sign
        for pool in (cache.k, cache.v):
            raw = pool.view(torch.uint8)
            for j in range(table.shape[1]):
                raw[int(table[0, j])][:, hide[j * bs:(j + 1) * bs].cuda()] = code
        got = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx_len.cuda(), q_start.cuda(), phase=phase, lse=True,
                                 cap=cap, scale=u * cap / top, first=first.cuda(), last=last.cuda())
        torch.cuda.synchronize()
        lci.get_device_status()
        seen.append([t.clone() for t in got])
    # NaN codes of V inside the context make the tile schedule compute rows again: those are as exact, not the same bits
    alike = seen if phase == "decode" else [seen[0], seen[2], seen[3]]
    for other in alike[1:]:
        assert torch.equal(other[0], alike[0][0]) and torch.equal(other[1], alike[0][1])
    assert torch.isfinite(seen[1][0]).all()


@pytest.mark.parametrize("S,topk,NB", [(1, 32, 3), (1, 5, 1), (40, 70, 8), (700, 33, 1100), (3, 256, 40)])
def test_block_weights_add_every_repeat_of_an_id(S, topk, NB):
    """Rows that hold a block more than once: each entry counts, and a repeat of the call gives the same bits."""
    g = torch.Generator().manual_seed(8)
    H = 2
    ids = torch.randint(-1, NB, (2, S, topk), generator=g).to(torch.int32)
    ids[0, 0] = NB - 1  # one block everywhere
    mass = torch.rand(2, S, H, topk, generator=g)
    weight = torch.rand(2, NB, generator=g)
    got = lci.block_weight_update(weight.cuda(), ids.cuda(), mass.cuda(), decay=0.5)
    torch.cuda.synchronize()
    lci.get_device_status()
    want = ref.weight_update(weight, ids, mass, 0.5)
    # fp32 sums of at most n addends of H masses each, one rounding of the total
    n = max(int(torch.bincount(ids[b][ids[b] >= 0].long().flatten()).max()) for b in range(2))
    assert ((got.cpu().double() - want).abs() <= want * 2.0 ** -24 * (H + 2 + n) + 1e-30).all()
    for _ in range(5):
        assert torch.equal(got, lci.block_weight_update(weight.cuda(), ids.cuda(), mass.cuda(), decay=0.5))


@pytest.mark.parametrize("shape,phase", [(SHAPES[5], "prefill"), (SHAPES[5], "decode"), (SHAPES[10], "auto")])
def test_v_scales_below_the_floor_count_as_the_floor(shape, phase):
    """In every schedule, and in rows that the tile schedule computes again (here
    for a NaN in another channel)."""
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(shape, 170)
    k, v, ks, vs = cpu
    vs.fill_(2.0 ** -70)
    floor = torch.full_like(vs, 2.0 ** -60)
    clean = v.clone()
    v.view(torch.uint8)[int(table[0, 0]), 0, 0, 3] = 0x7F
    cache = lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs)))
    bt = lci.create_block_table(table.cuda(), cache.k)
    out = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx_len.cuda(), q_start.cuda(), phase=phase).cpu().double()
    lci.get_device_status()
    ro, _, _, sizes = ref.attend(q, k.float(), clean.float(), ks, floor, table, bs, ids, ctx_len, q_start)
    # in units of the floor: 1e-30 of out_tolerance is far above these values
    tol = ref.out_tolerance(ro * 2.0 ** 60, (sizes[0], sizes[1] * 2.0 ** 60), q.dtype, q.shape[3],
                            24 if q.dtype == torch.float32 else 8) * 2.0 ** -60
    keep = torch.arange(q.shape[3]) != 3
    assert ((out - ro).abs() <= tol)[..., keep].all()


@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[10], (torch.float32, 1, 4, 70, 1, 9, 64, 16, 5)])
def test_masses_of_rows_that_meet_a_nan(shape):
    """A NaN among the attended keys makes the mass of every attended block of the
    row NaN, a block whose only token it is among them; other rows are what they
    are without it."""
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(shape, 180)
    k, v, ks, vs = cpu
    B, S = q.shape[:2]
    n = int(ctx_len[0])
    last = (n - 1) // bs
    for s in range(S):  # each row: the last block (one NaN in it), a hole, others
        ids[0, s] = -1
        ids[0, s, 0], ids[0, s, -1] = last, 0
    ids[0, 0, 0] = -1  # a row that does not select the block
    ctx_len[0] = last * bs + 1  # and only one token of it is attended: the NaN
    q_start[0] = int(ctx_len[0]) - 1
    clean = k.clone()
    k.view(torch.uint8)[int(table[0, last]), :, 0, 5] = 0x7F
    out = []
    for kk in (k, clean):
        cache = lci.Q8Cache.wrap(*(t.cuda() for t in (kk, v, ks, vs)))
        bt = lci.create_block_table(table.cuda(), cache.k)
        got = lci.sparse_attn_q8(q.cuda(), cache, bt, ids.cuda(), ctx_len.cuda(), q_start.cuda(), phase="decode", lse=True, mass=True)
        torch.cuda.synchronize()
        lci.get_device_status()
        out.append([t.cpu() for t in got])
    (o, l, m), (o2, l2, m2) = out
    hit = torch.zeros(B, S, dtype=torch.bool)
    hit[0, 1:] = True
    assert o[hit].isnan().all() and l[hit].isnan().all()
    assert (m2[hit] != 0).any() and m[hit][m2[hit] != 0].isnan().all()
    assert torch.equal(o[~hit], o2[~hit]) and torch.equal(m[~hit], m2[~hit])


@pytest.mark.parametrize("times", [1, 4, 16, 128])
@pytest.mark.parametrize("S,topk,G,bs,cap", [(2048, 16, 16, 64, 0.0), (2048, 8, 8, 128, 0.0), (3000, 16, 4, 64, 20.0)])
def test_a_prompt_takes_the_tile_schedule_in_tables_of_any_length(S, topk, G, bs, cap, times):
    """The schedules round weights differently: equal bits tell which one ran."""
    g = torch.Generator().manual_seed(190)
    cache, table, cpu = filled_cache(1, 1, bs, 128, [S], 191)
    nb = table.shape[1]
    wide = torch.full((1, min(nb * times, 16384)), -1, dtype=torch.int32)
    wide[:, :nb] = table
    q = torch.randn(1, S, G, 128, generator=g).to(torch.bfloat16).cuda()
    ids = torch.rand(S, nb, generator=g)
    ids[torch.arange(nb)[None] * bs > torch.arange(S)[:, None]] = -1.0  # blocks behind the query
    best = ids.topk(topk, dim=1)
    ids = torch.where(best.values >= 0, best.indices, -1).to(torch.int32)[None].cuda()
    bt = lci.create_block_table(wide.cuda(), cache.k)
    ctx, p0 = torch.tensor([S], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    out = {ph: lci.sparse_attn_q8(q, cache, bt, ids, ctx, p0, cap=cap, phase=ph) for ph in ("auto", "prefill", "decode")}
    torch.cuda.synchronize()
    lci.get_device_status()
    assert torch.equal(out["auto"], out["prefill"]) and not torch.equal(out["auto"], out["decode"])


@pytest.mark.parametrize("shape,phase", [(SHAPES[5], "prefill"), (SHAPES[5], "decode"), (SHAPES[0], "decode"), (SHAPES[10], "auto")])
def test_v_scales_at_the_largest_distance(shape, phase):
    """Blocks whose v scales are 2^96 apart: the softmax itself does not see them."""
    q, cache, table, cpu, bs, ids, ctx_len, q_start = attention_inputs(shape, 200)
    k, v, ks, vs = cpu
    vs.copy_(torch.where(torch.arange(len(vs)) % 2 == 0, 2.0 ** 48, 2.0 ** -48)[:, None].expand_as(vs))
    cache = lci.Q8Cache.wrap(*(t.cuda() for t in (k, v, ks, vs)))
    check_attention(q, cache, table, (k, v, ks, vs), bs, ids, ctx_len, q_start, phase=phase, mass=phase != "prefill",
                    p_bits=8 if phase == "prefill" else 11)
