"""The serving operators at the edges of their ranges, on the GPU against 64-bit definitions."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.serving_helpers import Pool, check_close  # noqa: E402
from tests.test_gpu_serving import run_prefix, run_prompt  # noqa: E402

FMTS = ["q8_0", "q4_0", "lut4", "nvfp4"]


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def fill(pool, k, v):
    """Write K and V [positions, 1, D] into slots 0 .. and read the cache's values back."""
    pool.cache.write(dev(k, np.float16), dev(v, np.float16), dev(np.arange(len(k))))
    torch.cuda.synchronize()
    pool.k, pool.v = pool.values("k"), pool.values("v")


# ------------------------------------------------------------------ small weights

# Weights enter the product with V in fp16 as 2^7 times their share of the maximum: steps of
# 2^-24, so each is off by at most 2^-25 / 2^7 = 2^-32 of the largest.  Pool.attend allows 2^-26
# per position; here the difference is the point.
STEP, POOL_STEP = 2.0 ** -32, 2.0 ** -26


def one_strong_key(fmt, n):
    """n positions: K 0 but for one key whose score is 26.3 binary orders above theirs, where V is
    0; V 1 elsewhere.  The answer is what the many small weights sum to."""
    D, gap = 64, 26.3
    pool = Pool(fmt, D, 1, 64, -(-n // 64), seed=40)
    k, v = np.zeros((n, 1, D), dtype=np.float16), np.ones((n, 1, D), dtype=np.float16)
    k[100], v[100] = 1.0, 0.0
    fill(pool, k, v)
    # the key as the cache holds it, so that the gap is what it should be in every format
    ones = np.ones((1, D))
    if fmt == "lut4":
        from oracle import quant as OQ
        ones = OQ.rotate_f64(ones, pool.signs)
    q1 = gap * math.log(2) * math.sqrt(D) / float(ones[0] @ pool.k[100, 0])
    return pool, q1


def tight(pool, q, n, half):
    """Pool.attend's answer and bound, with the steps of the weights as they are."""
    want, bound = pool.attend(q, np.arange(n), 1 / math.sqrt(pool.D))
    v = np.abs(pool.v[:n]).max()
    term = n * v * (math.sqrt(pool.D) if pool.fmt == "lut4" else 1.0)
    if pool.fmt == "lut4":
        # all small weights are equal and so is V: their rounding scales one vector, which is
        # rotated back as a whole
        from oracle import quant as OQ
        v = np.abs(OQ.unrotate_f64(pool.v[0], pool.signs)).max()
    bound = bound - term * POOL_STEP + n * v * STEP
    # what a lost tail would change has to stand out
    assert np.abs(want).min() > 1.5 * bound.max()
    return want, bound


@pytest.mark.parametrize("fmt", FMTS)
def test_prompt_small_weights_are_not_lost(fmt):
    # as many rows as keep a unit's positions in one piece; all rows are the same
    n, tokens, G = 32000, 4800, 8
    pool, q1 = one_strong_key(fmt, n)
    q = np.full((tokens, G, 64), q1, dtype=np.float16)
    out = pool.cache.prompt_attention(dev(q, np.float16), dev([0, tokens]), dev([n]), n, dev([np.arange(n // 64)]), n // 64,
                                      causal=False)
    want, bound = tight(pool, q[0], n, False)
    for i in (0, 77, tokens - 1):
        check_close(out[i].cpu().numpy(), want, bound, False)


@pytest.mark.parametrize("fmt", FMTS)
def test_prefix_small_weights_are_not_lost(fmt):
    # 1024 requests of 8 heads: 32 row tiles, four pieces of 8000 positions
    n, B, G = 32000, 1024, 8
    pool, q1 = one_strong_key(fmt, n)
    q = np.full((B, G, 64), q1, dtype=np.float16)
    out = pool.cache.prefix_attention(dev(q, np.float16), dev([np.arange(n // 64)]), dev([n]), n, dev([0] * B), 0,
                                      dev([[0]] * B), 1)
    want, bound = tight(pool, q[0], n, False)
    for i in (0, 500, B - 1):
        check_close(out[i].cpu().numpy(), want, bound, False)


# ------------------------------------------------------------------ a stream given by its handle

@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["prompt", "prefix", "decode"])
def test_explicit_stream_takes_no_memory_of_another(op, raw):
    """With stream=, the output and the workspace come from that stream's memory: a block that was
    freed on the current one may still be in use there."""
    pool = Pool("q4_0", 64, 1, 64, 40, seed=49)
    q = dev(pool.queries(64, 8), np.float16)
    tab, lens = dev([np.arange(40)]), dev([2500])
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    many = dev([2500] * 64), dev(np.tile(np.arange(40), (64, 1)))
    call = {"prompt": lambda **kw: pool.cache.prompt_attention(q, dev_off, lens, 2560, tab, 40, **kw),
            "prefix": lambda **kw: pool.cache.prefix_attention(q, tab, lens, 2560, zero, 0, own, 1, **kw),
            "decode": lambda **kw: pool.cache.attention(q, many[0], 2560, many[1], 40, tau=0.0, **kw)}[op]
    dev_off, zero, own = dev([0, 64]), dev([0] * 64), dev([[0]] * 64)
    want = call()
    torch.cuda.synchronize()
    fresh = Pool("q4_0", 64, 1, 64, 40, seed=49)
    pool.cache, old = fresh.cache, pool.cache
    # every block that the calls could want, freed on the current stream
    sizes = [want.numel() * 4] + [t.numel() for t in (old._ws, *old._ws_rows.values()) if t is not None]
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    spans = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
    del blocks
    torch.cuda.synchronize()
    out = call(stream=s)
    side.synchronize()
    mine = [out] + [t for t in (pool.cache._ws, *pool.cache._ws_rows.values()) if t is not None]
    for t in mine:
        assert not any(a < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < b for a, b in spans)
    if op == "decode":   # its atomics' order may change the last bits
        torch.testing.assert_close(out, want, rtol=0, atol=1e-5)
    else:
        assert torch.equal(out, want)
    assert pool.cache.device_flags() == 0


# ------------------------------------------------------------------ captured calls

def test_flags_of_captured_calls():
    """Warm-up on one stream, capture on torch's own: the flags of every replay stay until they
    are read, in the first graph and in a second one."""
    import quantized_kv_cache_split_b200 as K
    pool = Pool("q8_0", 64, 1, 64, 10, seed=45)
    q, lens = dev(pool.queries(4, 4), np.float16), dev([600])
    off, table = dev([0, 4]), dev([np.arange(10)])
    out = torch.zeros(4, 4, 64, device="cuda")
    call = lambda: pool.cache.prompt_attention(q, off, lens, 640, table, 10, out=out)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    want = out.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    assert pool.cache.device_flags() == 0
    for g in reversed(graphs):                                  # the second before the first
        out.zero_()
        g.replay()
        assert torch.equal(out, want) and pool.cache.device_flags() == 0
    lens.fill_(-1)
    graphs[1].replay()
    lens.fill_(600)
    for g in graphs:                                            # clean replays do not hide it
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert pool.cache.device_flags() == K.KVQ_FLAG_BAD_SEQLEN


def test_captured_calls_have_their_own_workspace():
    """Graphs replayed at once on two streams, beside eager calls on a third that need a larger
    workspace: each gives what it gives alone."""
    pool = Pool("q4_0", 64, 1, 64, 60, seed=46)
    table = dev([np.arange(60)])
    qs = [dev(pool.queries(n, 8), np.float16) for n in (3, 5, 90)]
    outs = [torch.zeros(q.shape, device="cuda") for q in qs]
    lens = [dev([n]) for n in (3800, 3000, 2500)]
    offs = [dev([0, q.shape[0]]) for q in qs]
    call = lambda i: pool.cache.prompt_attention(qs[i], offs[i], lens[i], 3840, table, 60, out=outs[i])  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(2):
            call(i)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs[:2]]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g, stream=side):
            call(i)
    with torch.cuda.stream(side):
        call(2)
    torch.cuda.synchronize()
    want.append(outs[2].clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(side):
            call(2)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert pool.cache.device_flags() == 0


# ------------------------------------------------------------------ calls without work

def test_calls_without_work():
    import quantized_kv_cache_split_b200 as K
    pool = Pool("q4_0", 64, 2, 64, 4, seed=44)
    c, none = pool.cache, torch.zeros(0, dtype=torch.int32, device="cuda")
    q0 = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda")
    table = dev([[0, 1], [2, 3]])
    assert c.prompt_attention(q0, dev([0, 0, 0]), dev([100, 5]), 128, table, 2).shape == (0, 4, 64)     # no new tokens
    assert c.prompt_attention(q0, dev([0]), none, 128, none.view(0, 2), 2).shape == (0, 4, 64)          # no requests
    pad = torch.full((3, 4, 64), 2.0, device="cuda")
    c.prompt_attention(dev(pool.queries(3, 4), np.float16), dev([0]), none, 128, none.view(0, 2), 2, out=pad)
    assert (pad == 2.0).all()                                                                           # padding alone
    assert c.prefix_attention(q0, dev([[0, 1]]), dev([100]), 128, none, 64, none.view(0, 2), 2).shape == (0, 4, 64)
    p = K.PagePlanner(0, 64, 4, 2, 8)
    assert (p.slots == -1).all()                                  # before a step nothing has a slot
    p.step(none, none.view(0, 2), p.seq_lens, dev([0, 1, 2, 3]), p.free_count)
    assert (p.slots == -1).all()
    p = K.PagePlanner(2, 64, 4, 2, 0)                             # room for no token
    p.free_count.fill_(4)
    p.step(dev([0, 0]), table, p.seq_lens, dev([0, 1, 2, 3]), p.free_count)
    assert p.device_flags() == 0 and c.device_flags() == 0


# ------------------------------------------------------------------ memory that a cache keeps

def test_workspaces_do_not_pile_up():
    # prompts of rising length: the rotated format's partials are the largest
    pool = Pool("lut4", 64, 1, 64, 40, seed=48)
    q = dev(pool.queries(1600, 8), np.float16)
    table = dev([np.arange(40)])
    out = torch.zeros(1600, 8, 64, device="cuda")
    torch.cuda.synchronize()
    start = torch.cuda.memory_allocated()
    for n in range(1200, 1602, 2):
        pool.cache.prompt_attention(q[:n], dev([0, n]), dev([n]), n, table, 40, out=out[:n])
    torch.cuda.synchronize()
    import quantized_kv_cache_split_b200 as K
    assert torch.cuda.memory_allocated() - start < 2 * K.kvq_prompt_workspace_size(pool.cache.desc, 1600, 8, 1, 1600)
    assert len(pool.cache._rows_bytes) <= 64


# ------------------------------------------------------------------ lengths above a bound of zero

def test_prefix_lengths_above_zero_bounds_set_flags():
    import quantized_kv_cache_split_b200 as K
    pool = Pool("q8_0", 64, 1, 64, 8, seed=47)
    q, tab, own = dev(pool.queries(3, 2), np.float16), dev([[0, 1], [2, 3]]), dev([[4], [5], [6]])
    call = lambda c, off, plens, pmax, lens, omax: c.prefix_attention(  # noqa: E731
        q, tab, dev(plens), pmax, dev(lens), omax, own, 1, group_offsets=dev(off))
    for off, plens, pmax, lens, omax, flag in (
            ([0, 2, 3], [100, 7], 128, [5, 0, 9], 64, 0), ([0, 2, 3], [0, 0], 0, [5, 0, 9], 64, 0),
            ([0, 2, 3], [0, 0], 0, [0, 0, 0], 0, 0),
            ([0, 2, 3], [0, 5], 0, [5, 0, 9], 64, K.KVQ_FLAG_BAD_SEQLEN),       # a prefix above a bound of 0
            ([0, 3, 3], [0, -1], 0, [5, 0, 9], 64, K.KVQ_FLAG_BAD_SEQLEN),      # of a group without requests
            ([0, 2, 1], [0, 0], 0, [5, 0, 9], 64, K.KVQ_FLAG_BAD_SEQLEN),       # offsets that fall
            ([0, 2, 4], [0, 0], 0, [5, 0, 9], 64, K.KVQ_FLAG_BAD_SEQLEN),       # and leave the batch
            ([-1, 2, 3], [0, 0], 0, [5, 0, 9], 64, K.KVQ_FLAG_BAD_SEQLEN),
            ([0, 2, 3], [100, 7], 128, [0, 5, 0], 0, K.KVQ_FLAG_BAD_SEQLEN),    # own positions above a bound of 0
            ([0, 2, 3], [0, 0], 0, [0, 0, -1], 0, K.KVQ_FLAG_BAD_SEQLEN)):
        cache = K.QuantizedKVCache("q8_0", 64, 1, 64, 8)
        call(cache, off, plens, pmax, lens, omax)
        assert cache.device_flags() == flag, (off, plens, pmax, lens, omax)


# ------------------------------------------------------------------ NaN in positions that are seen

def set_nan(pool, position, plane):
    """A NaN scale at a slot, in every format (0xff bytes: fp16, e4m3 and fp32 NaN)."""
    t = getattr(pool.cache, plane)
    t[position // pool.ps, :, position % pool.ps].view(torch.uint8).fill_(0xff)
    torch.cuda.synchronize()


@pytest.mark.parametrize("plane", ["k_scales", "v_scales"])
@pytest.mark.parametrize("fmt", FMTS)
# one piece of one row tile, of two; pieces that the merge joins; a single position
@pytest.mark.parametrize("n,tokens,at", [(400, 20, 333), (400, 20, 150), (400, 200, 3), (400, 200, 300), (5000, 3, 4700), (1, 1, 0)])
def test_prompt_nan_reaches_every_row_that_sees_it(fmt, plane, n, tokens, at):
    pool = Pool(fmt, 64, 1, 64, 80, seed=41)
    q = dev(pool.queries(tokens, 4), np.float16)
    args = (dev([0, tokens]), dev([n]), n, dev([np.arange(80)]), 80)
    clean = pool.cache.prompt_attention(q, *args)
    set_nan(pool, at, plane)
    out = pool.cache.prompt_attention(q, *args)
    sees = torch.arange(tokens, device="cuda") + n - tokens >= at
    assert torch.isnan(out[sees]).all()
    if plane == "k_scales":   # (a V that is not finite may reach tokens before it)
        assert torch.equal(out[~sees], clean[~sees])


@pytest.mark.parametrize("plane", ["k_scales", "v_scales"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_prefix_nan_reaches_every_request_that_sees_it(fmt, plane, where):
    pool = Pool(fmt, 64, 1, 64, 40, seed=42)
    q = dev(pool.queries(3, 4), np.float16)
    args = (q, dev([np.arange(30)]), dev([1900]), 1920, dev([100, 0, 70]), 128, dev([[30, 31], [32, 33], [34, 35]]), 2)
    clean = pool.cache.prefix_attention(*args)
    assert torch.isfinite(clean).all()
    set_nan(pool, 1234 if where == "prefix" else 34 * 64 + 69, plane)
    out = pool.cache.prefix_attention(*args)
    if where == "prefix":
        assert torch.isnan(out).all()
    else:
        assert torch.isnan(out[2]).all() and torch.equal(out[:2], clean[:2])


# ------------------------------------------------------------------ scores far beyond ordinary ones

@pytest.mark.parametrize("sm_scale", [1.0, 0.1, -0.1, 0.002])
@pytest.mark.parametrize("tokens", [3, 40, 200])
def test_prompt_huge_scores(tokens, sm_scale):
    # queries and keys of thousands.  Keys are equal within a stretch (so their scores are too) and
    # the stretches' scores lie thousands apart: the answer is the mean of V over the best stretch
    # that a row sees.  With sm_scale 1 the scores pass 2^27 (up to 6e8): right or not finite.
    n, D, G = 700, 64, 4
    pool = Pool("q8_0", D, 1, 64, 11, seed=43)
    rng = pool.rng
    level = np.repeat([508.0, 1016.0, 254.0, 2032.0, 127.0, 1524.0, 63.5], 100)   # 127 * scale, exact
    k = np.broadcast_to(level[:, None, None], (n, 1, D)).astype(np.float16)
    v = rng.integers(-127, 128, (n, 1, D)).astype(np.float16)
    v[:, :, 0::32] = 127.0                                                   # scale 1: exact
    fill(pool, k, v)
    assert np.array_equal(pool.v[:n], v.astype(np.float64))
    q = (rng.uniform(0.5, 1.5, (tokens, G, 1)) * rng.integers(500, 3000, (tokens, G, 1))
         * rng.choice([-1.0, 1.0], (tokens, G, 1)) * np.ones(D)).astype(np.float16)
    out = pool.cache.prompt_attention(dev(q, np.float16), dev([0, tokens]), dev([n]), n, dev([np.arange(11)]), 11,
                                      sm_scale=sm_scale).cpu().numpy().astype(np.float64)
    for i in range(tokens):
        seen = n - tokens + i + 1
        for h in range(G):
            s = level[:seen] * np.sign(q[i, h, 0]) * np.sign(sm_scale)
            want = pool.v[:seen][s == s.max(), 0].mean(0)
            # equal weights, whose sum is taken before their common rounding to fp16 (2^-11), and
            # fp32 sums
            right = np.abs(out[i, h] - want).max() <= 127 * (2.0 ** -11 + 2.0 ** -16)
            assert right or sm_scale == 1.0 and not np.isfinite(out[i, h]).all(), (i, h)
    assert pool.cache.device_flags() == 0


# ------------------------------------------------------------------ flags of steps on another stream

def test_planner_flags_wait_for_the_steps_stream():
    import quantized_kv_cache_split_b200 as K
    p = K.PagePlanner(2, 64, 8, 2, 16)
    table, free, count = dev([[0, -1], [1, -1]]), dev(np.arange(8)), dev([4])
    new, lens = dev([1, 1]), dev([5, 7])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000)
        p.step(new, table, lens, free, count)        # the kernels are loaded now
    lens[1] = -1
    torch.cuda.synchronize()
    assert p.device_flags() == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)               # a tenth of a second
        p.step(new, table, lens, free, count)
    assert p.device_flags() == K.KVQ_FLAG_BAD_SEQLEN


# ------------------------------------------------------------------ many groups, split along their positions

@pytest.mark.parametrize("groups", [33, 40, 70])
@pytest.mark.parametrize("fmt", ["q8_0", "lut4"])
def test_prompt_many_groups_of_several_pieces(fmt, groups):
    # more groups than lanes of a warp, few enough units that positions are split: the fixed chunk,
    # the search for a block's group and the merge over the pieces; long requests beside short ones,
    # requests without tokens and without positions
    import quantized_kv_cache_split_b200 as K
    pool = Pool(fmt, 64, 1, 64, 420, seed=50)
    old, new = pool.rng.integers(0, 130, groups), pool.rng.integers(0, 4, groups)
    for b, n in ((0, 3000), (groups // 2, 1025), (groups - 2, 2047), (groups - 1, 1500)):
        old[b] = n
    new[[0, groups // 2, groups - 1]] = 2, 70, 1
    old[5], new[5] = -1, 2                     # the first of its tokens sees nothing
    old[6], new[6] = 0, 0
    rows, longest = int(new.sum()) + 3, int((old + new).max())
    one = 256 + rows * 4 * (64 + 2) * 4        # a workspace of one piece
    assert K.kvq_prompt_workspace_size(pool.cache.desc, rows, 4, groups, longest) > one
    run_prompt(pool, 4, old, new, pad=3, causal=False, half=False, poison=False)
    run_prompt(pool, 4, old, new, pad=3)       # (leaves NaN in the slots of no request)


@pytest.mark.parametrize("fmt", ["q4_0", "lut4"])
def test_prefix_many_groups_of_several_pieces(fmt):
    import quantized_kv_cache_split_b200 as K
    pool = Pool(fmt, 64, 1, 64, 420, seed=51)
    groups = 40
    prefix, sizes = pool.rng.integers(0, 130, groups), pool.rng.integers(0, 3, groups)
    prefix[[0, 7, 20, 39]] = 3000, 0, 1500, 2047
    sizes[[0, 7, 20, 39]] = 3, 2, 40, 1
    B = int(sizes.sum())
    own = pool.rng.integers(0, 60, B)
    d = pool.cache.desc
    # more than one piece of the prefixes beside the own part's (that of a short prefix has one)
    assert K.kvq_prefix_workspace_size(d, B, 4, groups, 3000, 60) > K.kvq_prefix_workspace_size(d, B, 4, groups, 100, 60)
    run_prefix(pool, 4, [int(n) for n in prefix], [int(n) for n in sizes], [int(n) for n in own])


# ------------------------------------------------------------------ bad pages, lengths and offsets of a prefix decode

@pytest.mark.parametrize("groups", [2, 40])
def test_prefix_bad_pages_and_lengths_set_flags(groups):
    """In bounds whatever the tables hold: the flags say so (a search finds the group of more than
    32)."""
    import quantized_kv_cache_split_b200 as K
    pool = Pool("q8_0", 64, 1, 64, 8, seed=52)
    B = groups + 1
    q = dev(pool.queries(B, 2), np.float16)
    at = groups - 1                                     # the group and the request that are wrong
    for what, flag in (("nothing", 0), ("prefix page", K.KVQ_FLAG_BAD_PAGE), ("prefix page -1", K.KVQ_FLAG_BAD_PAGE),
                       ("own page", K.KVQ_FLAG_BAD_PAGE), ("own page -1", K.KVQ_FLAG_BAD_PAGE),
                       ("prefix long", K.KVQ_FLAG_BAD_SEQLEN), ("prefix -1", K.KVQ_FLAG_BAD_SEQLEN),
                       ("own long", K.KVQ_FLAG_BAD_SEQLEN), ("own -1", K.KVQ_FLAG_BAD_SEQLEN),
                       ("offset -1", K.KVQ_FLAG_BAD_SEQLEN), ("offset falls", K.KVQ_FLAG_BAD_SEQLEN),
                       ("offset leaves", K.KVQ_FLAG_BAD_SEQLEN)):
        ptab, plens = np.tile([0, 1, 2], (groups, 1)), np.full(groups, 150)
        tab, lens, off = np.tile([3, 4], (B, 1)), np.full(B, 100), np.arange(groups + 1)
        off[-1] = B
        if "prefix page" in what:
            ptab[at, 1] = -1 if "-1" in what else 8
        elif "own page" in what:
            tab[at, 1] = -1 if "-1" in what else 8
        elif "prefix" in what:
            plens[at] = -1 if "-1" in what else 193
        elif "own" in what:
            lens[at] = -1 if "-1" in what else 129
        elif what == "offset -1":
            off[0] = -1
        elif what == "offset falls":
            off[at] = B - 3 if groups > 2 else 0
            off[at - 1] = B - 2 if groups > 2 else 1
        elif what == "offset leaves":
            off[-1] = B + 1
        cache = K.QuantizedKVCache("q8_0", 64, 1, 64, 8)
        out = cache.prefix_attention(q, dev(ptab), dev(plens), 192, dev(lens), 128, dev(tab), 2, group_offsets=dev(off))
        assert out.shape == q.shape and cache.device_flags() == flag, what


# ------------------------------------------------------------------ a captured plan of two launches

def test_captured_large_plan_replays():
    # more than 65,536 slots: the slots come from a second launch, scheduled early; the state stays
    # on the GPU and moves on with each replay
    import quantized_kv_cache_split_b200 as K
    from tests.serving_helpers import plan_reference
    B, ps, mp, num_pages, cap = 40, 64, 30, 1300, 70001
    p = K.PagePlanner(B, ps, num_pages, mp, cap)
    rng = np.random.Generator(np.random.PCG64(53))
    table, free = torch.full((B, mp), -1, dtype=torch.int32, device="cuda"), dev(rng.permutation(num_pages))
    p.free_count.fill_(num_pages)
    new = dev(rng.integers(0, 300, B))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.step(new, table, p.seq_lens, free, p.free_count)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.step(new, table, p.seq_lens, free, p.free_count)
    for turn in range(5):
        new.copy_(dev(np.where(rng.random(B) < 0.3, -1, rng.integers(0, 300, B))))
        was = [t.cpu().numpy() for t in (p.seq_lens, new, free, p.free_count, table)]
        want = plan_reference(was[0], was[1], was[2], int(was[3][0]), was[4], ps, cap)
        graph.replay()
        assert p.device_flags() == 0
        assert np.array_equal(table.cpu().numpy(), want["table"])
        assert np.array_equal(free.cpu().numpy()[:len(want["stack"])], want["stack"])
        for name, t in (("lens", p.seq_lens), ("offsets", p.token_offsets), ("slots", p.slots), ("positions", p.positions)):
            assert np.array_equal(t.cpu().numpy(), want[name]), (turn, name)


# ------------------------------------------------------------------ one rounding of a K or V value

U = 2.0 ** -11 * (1 + 2.0 ** -9)   # half a step of fp16, and what fp32 adds


def requests_of(fmt, n, positions, seed):
    """n requests of a page each with the given K and V rows [n, positions, 1, D]."""
    pool = Pool(fmt, 64, 1, 64, n, seed=seed)
    return pool, np.arange(n)[:, None] * 64 + np.arange(positions)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "nvfp4"])
@pytest.mark.parametrize("op", ["prompt", "own"])
def test_values_are_rounded_once(fmt, op):
    # a single position has weight 1 exactly: the answer is V as it enters the product
    n = 300
    pool, slots = requests_of(fmt, n, 1, 54)
    q, lens, table = dev(pool.queries(n, 2), np.float16), dev([1] * n), dev(np.arange(n).reshape(n, 1))
    if op == "prompt":
        out = pool.cache.prompt_attention(q, dev(np.arange(n + 1)), lens, 64, table, 1)
    else:
        out = pool.cache.prefix_attention(q, dev([[0]]), dev([0]), 64, lens, 64, table, 1)
    want = np.repeat(pool.v[slots[:, 0]], 2, 1)
    err = np.abs(out.cpu().numpy() - want)
    assert (err <= np.abs(want) * U + 2.0 ** -24).all(), float((err / np.maximum(np.abs(want) * U, 1e-30)).max())


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "nvfp4"])
def test_keys_are_rounded_once(fmt):
    # two positions, K 0 and V 0 at the first, K the same c in every dimension and V 1 at the second:
    # the answer is the second's weight, 1 / (1 + e^-s), from which the score's error shows.  The
    # roundings of equal K values are equal and add up.
    n, D = 300, 64
    pool, slots = requests_of(fmt, n, 2, 55)
    rng = pool.rng
    k = np.zeros((n, 2, 1, D), dtype=np.float16)
    k[:, 1] = rng.uniform(0.5, 2.0, (n, 1, 1))
    k[:, 1, 0, ::16] *= rng.uniform(1.0, 3.0, (n, 1))          # other block and vector scales
    v = np.zeros((n, 2, 1, D), dtype=np.float16)
    v[:, 1] = 1.0
    pool.cache.write(dev(k.reshape(-1, 1, D), np.float16), dev(v.reshape(-1, 1, D), np.float16), dev(slots.reshape(-1)))
    torch.cuda.synchronize()
    pool.k, pool.v = pool.values("k"), pool.values("v")
    q = np.full((n, 1, D), 0.25, dtype=np.float16)
    out = pool.cache.prompt_attention(dev(q, np.float16), dev(np.arange(n + 1)), dev([2] * n), 64,
                                      dev(np.arange(n).reshape(n, 1)), 1).cpu().numpy().astype(np.float64)
    s = (0.25 / math.sqrt(D)) * pool.k[slots[:, 1], 0].sum(-1)
    w = 1 / (1 + np.exp(-s))
    got = (out[:, 0] / pool.v[slots[:, 1], 0]).mean(-1)
    # V is rounded too (its error is the same in every dimension); w' = w (1 - w)
    assert (np.abs(got - w) <= w * (1 - w) * s * U * (1 + s * U) + w * 2.0 ** -20 + w * np.abs(
        np.float64(np.float16(pool.v[slots[0, 1], 0, 0] / 2)) * 2 - pool.v[slots[0, 1], 0, 0])).all()
