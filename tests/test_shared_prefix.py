"""fd_decode_shared_prefix: attention of rows that share prompts, against the definition in 64 bits.

Tolerances.  A score is a sum of d products in f32, off by at most
delta = d 2^-23 max_t sum_i |q_i k_ti| / sqrt(d) (d roundings of partial sums, each counted a
whole step).  So exp(score) is off by 2 delta relative and lse by delta, plus the base-2
exponential's and logarithm's own errors (2^-20).  With A = sum_t w_t |v_t| the output is off
by (2 delta + 2^-18) A from that; from rounding each weight to bf16 by 2^-8 A (bf16 and FP8
caches); from f32 sums over n keys by n 2^-24 A; and from its own rounding by half a step.
"""
import math

import pytest
import torch

fd = pytest.importorskip("decode_attention_05_gb300")

INVALID, UNSUPPORTED, WS_SMALL = 1, 2, 3
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------------ refusals (no GPU)


def _bf(*shape):
    return torch.zeros(shape, dtype=BF)


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def _aligned(n):
    """n bytes at a 256-byte border, as device allocations have."""
    t = torch.zeros(n + 256, dtype=torch.uint8)
    at = -t.data_ptr() % 256
    return t[at:at + n]


def _cpu_case(**over):
    a = dict(q=_bf(4, 8, 128), k_prefix=_bf(1, 2, 64, 128), v_prefix=_bf(1, 2, 64, 128),
             prefix_lens=_ints(60), k_cache=_bf(4, 2, 16, 128), v_cache=_bf(4, 2, 16, 128),
             seq_lens=_ints(1, 2, 3, 4), workspace=_aligned(1 << 20), stream=0)
    a.update(over)
    return a


def _f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(F8)


two = dict(k_prefix=_bf(2, 2, 64, 128), v_prefix=_bf(2, 2, 64, 128), prefix_lens=_ints(60, 5))
REFUSED = [
    ("prefix shapes", dict(v_prefix=_bf(1, 2, 32, 128)), INVALID),
    ("prefix heads", dict(k_prefix=_bf(1, 1, 64, 128), v_prefix=_bf(1, 1, 64, 128)), INVALID),
    ("prefix dtype", dict(k_prefix=torch.zeros(1, 2, 64, 128), v_prefix=torch.zeros(1, 2, 64, 128)), INVALID),
    ("two prefixes without groups", two, INVALID),
    ("q dtype", dict(q=torch.zeros(4, 8, 128)), INVALID),
    ("q heads", dict(q=_bf(4, 7, 128)), INVALID),
    ("rows of the cache", dict(k_cache=_bf(3, 2, 16, 128), v_cache=_bf(3, 2, 16, 128)), INVALID),
    ("head dim", dict(q=_bf(4, 8, 96), k_prefix=_bf(1, 2, 64, 96), v_prefix=_bf(1, 2, 64, 96),
                      k_cache=_bf(4, 2, 16, 96), v_cache=_bf(4, 2, 16, 96)), UNSUPPORTED),
    ("too many query rows", dict(q=_bf(4, 17, 8, 128)), UNSUPPORTED),
    ("group size", dict(q=_bf(4, 6, 128)), UNSUPPORTED),
    ("out dtype", dict(out=torch.zeros(4, 8, 128, dtype=torch.int32)), UNSUPPORTED),
    ("out shape", dict(out=_bf(4, 4, 128)), INVALID),
    ("misaligned out", dict(out=_bf(4 * 8 * 128 + 8)[1:-7].view(4, 8, 128)), INVALID),
    ("scales without fp8", dict(k_scale=torch.ones(2)), INVALID),
    ("fp8 head dim", dict(q=_bf(4, 8, 64), k_prefix=_f8(1, 2, 64, 64), v_prefix=_f8(1, 2, 64, 64),
                          k_cache=_f8(4, 2, 16, 64), v_cache=_f8(4, 2, 16, 64)), UNSUPPORTED),
    ("page size without a table", dict(page_size=16), INVALID),
    ("prefix page size", dict(page_size=12, prefix_table=torch.zeros(1, 4, dtype=torch.int32)), INVALID),
    ("prefix pool's page", dict(page_size=16, prefix_table=torch.zeros(1, 4, dtype=torch.int32)), INVALID),
    ("prefix table dtype", dict(page_size=64, prefix_table=torch.zeros(1, 4)), INVALID),
    ("overlapping out rows", dict(out=_bf(1, 8, 128).expand(4, 8, 128)), INVALID),
    ("misaligned workspace", dict(workspace=_aligned(1 << 20)[16:]), INVALID),
    ("prefix splits", dict(prefix_splits=-1), INVALID),
    ("splits", dict(num_splits=4097), INVALID),
    ("small workspace", dict(workspace=_aligned(4096)), WS_SMALL),
    ("prefix token rows overlap", dict(
        k_prefix=_bf(1, 2, 64, 128).as_strided((1, 2, 64, 128), (16384, 8192, 64, 1))), INVALID),
    ("options", dict(options=fd.FdOptions(9, 0, 0)), INVALID),
]


@pytest.mark.parametrize("name,over,status", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(name, over, status):
    with pytest.raises(fd.FdError) as e:
        fd.decode_attention_shared_prefix(**_cpu_case(**over))
    assert e.value.status == status


def test_binding_checks_host_visible_sizes():
    for over in (dict(seq_lens=_ints(1)), dict(prefix_lens=_ints(1, 2)), dict(group_start=_ints(0, 4, 4)),
                 dict(k_scale=torch.ones(3))):
        with pytest.raises(ValueError):
            fd.decode_attention_shared_prefix(**_cpu_case(**over))
    for over in (dict(prefix_lens=torch.ones(1)), dict(lse_out=torch.zeros(4, 8, 1)),
                 dict(seq_lens=torch.ones(4, dtype=torch.int64))):
        with pytest.raises(TypeError):
            fd.decode_attention_shared_prefix(**_cpu_case(**over))


def test_sizes():
    size = fd.shared_prefix_workspace_size
    assert size(0, 1, 8, 2, 128, 1, 64, 16) == 0 and size(4, 1, 8, 3, 128, 1, 64, 16) == 0
    assert size(4, 1, 8, 2, 128, 1, 0, 16) == 0 and size(4, 1, 8, 2, 128, 1, 64, 16, 4097) == 0
    own = fd.workspace_size(4, 8, 2, 128, 3)
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert size(4, 1, 8, 2, 128, 1, 640, 160, 5, 3) == up(up(up(own) + 32 * 5 * 4) + 32 * 5 * 128 * 4)
    assert fd.resolve_prefix_splits(4, 1, 8, 2, 1, 640, 7) == 7
    assert fd.resolve_prefix_splits(4, 1, 8, 2, 1, 640) >= 1


# ------------------------------------------------------------------ the definition, 64 bits


class Case:
    """Inputs on the CPU, `call` on the GPU, and the definition's (out, lse, tolerances)."""

    def __init__(self, dtype=BF, cache=None, d=128, Hq=8, Hkv=2, Q=1, groups=((3, 70),), own=(5, 0, 9),
                 page=0, own_page=None, behind=0, cap=None, seed=0, scale=1.0, poison=True, spikes=False):
        g = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        own_page = page if own_page is None else own_page
        self.Q, self.Hq, self.Hkv, self.d, self.page, self.dtype = Q, Hq, Hkv, d, page or own_page, dtype
        sizes, plens = [n for n, _ in groups], [x for _, x in groups]
        B, P = sum(sizes) + behind, len(groups)
        own = [own[b % len(own)] for b in range(B)]
        self.B, self.P = B, P
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q = (rnd(B, Q, Hq, d) * scale).to(dtype)
        self.ks = self.vs = None
        if cache == F8:
            self.ks, self.vs = torch.rand(Hkv, generator=g) + 0.5, torch.rand(Hkv, generator=g) + 0.5

        def cached(lens, page):
            """Dense [rows, Hkv, cap, d] in the cache's type, with its stored form."""
            most = max(max(lens), 1) if cap is None else cap
            if page:
                most = -(-most // page) * page
            k, v = rnd(len(lens), Hkv, most, d).to(BF), rnd(len(lens), Hkv, most, d).to(BF)
            if spikes:
                for r in range(len(lens)):
                    k[r, :, ::37] *= 12
            if dtype == F32:
                k, v = k.float() + 2.0 ** -12 * rnd(*k.shape), v.float() + 2.0 ** -12 * rnd(*v.shape)
            if poison:
                for r, n in enumerate(lens):
                    k[r, :, n:], v[r, :, n:] = math.nan, math.nan
            k, v = k.to(cache), v.to(cache)
            if not page:
                return k, v, k, v, None
            w = most // page
            bytes_ = lambda x: x.view(torch.uint8) if cache == F8 else x  # noqa: E731
            order = torch.randperm(len(lens) * w + 2, generator=g)[:len(lens) * w]
            pools = []
            for x in (k, v):
                pool = torch.full((len(lens) * w + 2, Hkv, page, d), math.nan, dtype=BF).to(cache)
                bytes_(pool)[order] = bytes_(x).unflatten(2, (w, page)).transpose(1, 2).flatten(0, 1)
                pools.append(pool)
            table = order.view(len(lens), w).to(torch.int32)
            for r, n in enumerate(lens):
                table[r, -(-n // page):] = -1
            return k, v, pools[0], pools[1], table

        self.kp, self.vp, self.kp_, self.vp_, self.pt = cached(plens, page)
        self.ko, self.vo, self.ko_, self.vo_, self.bt = cached(own, own_page)
        self.plens, self.own, self.sizes = plens, own, sizes
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + n)
        self.starts = _ints(*starts) if P > 1 or behind else None

    def args(self):
        gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
        q = self.q if self.Q > 1 else self.q[:, 0]
        return dict(q=gpu(q), k_prefix=gpu(self.kp_), v_prefix=gpu(self.vp_),
                    prefix_lens=gpu(_ints(*self.plens)), k_cache=gpu(self.ko_), v_cache=gpu(self.vo_),
                    seq_lens=gpu(_ints(*self.own)), group_start=gpu(self.starts),
                    prefix_table=gpu(self.pt), block_table=gpu(self.bt), page_size=self.page,
                    k_scale=gpu(self.ks), v_scale=gpu(self.vs))

    def exact(self, out_dtype=None):
        G, d = self.Hq // self.Hkv, self.d
        shape = (self.B, self.Q, self.Hq)
        out, tol = torch.zeros(*shape, d, dtype=torch.float64), torch.zeros(*shape, d, dtype=torch.float64)
        lse, ltol = torch.full(shape, -math.inf, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
        group = [i for i, n in enumerate(self.sizes) for _ in range(n)] + [None] * self.B
        step = torch.finfo(out_dtype or self.dtype).eps / 2
        weight = 0.0 if self.dtype == F32 else 2.0 ** -8
        for b in range(self.B):
            p = group[b]
            for h in range(self.Hq):
                g = h // G
                kk, vv = self.ko[b, g, :self.own[b]].double(), self.vo[b, g, :self.own[b]].double()
                n = 0
                if p is not None:
                    n = self.plens[p]
                    kk = torch.cat([self.kp[p, g, :n].double(), kk])
                    vv = torch.cat([self.vp[p, g, :n].double(), vv])
                if self.ks is not None:
                    kk, vv = kk * self.ks[g].double(), vv * self.vs[g].double()
                for j in range(self.Q):
                    m = n + max(0, min(self.own[b], self.own[b] - self.Q + 1 + j))
                    if m == 0:
                        continue
                    x = self.q[b, j, h].double()
                    s = kk[:m] @ x / math.sqrt(d)
                    delta = d * 2.0 ** -23 * float((kk[:m].abs() @ x.abs()).max()) / math.sqrt(d)
                    l = torch.logsumexp(s, 0)
                    w = (s - l).exp()
                    o, A = w @ vv[:m], w @ vv[:m].abs()
                    out[b, j, h], lse[b, j, h] = o, l
                    tol[b, j, h] = step * o.abs() + (weight + 2 * delta + 2.0 ** -18 + m * 2.0 ** -24) * A
                    ltol[b, j, h] = delta + 2.0 ** -20 + 2.0 ** -22 * abs(float(l))
        return out, tol, lse, ltol

    def check(self, out, lse, out_dtype=None, want=None):
        o, tol, l, ltol = want or self.exact(out_dtype)
        out, lse = out.double().cpu().view(o.shape), lse.double().cpu().view(l.shape)
        assert not torch.isnan(out).any() and not torch.isnan(lse).any()
        off = (out - o).abs() - tol
        assert bool((off <= 0).all()), "out off by %g over its tolerance" % float(off.max())
        none = torch.isinf(l)
        assert torch.equal(torch.isinf(lse) & (lse < 0), none)
        off = (lse - l).abs()[~none] - ltol[~none]
        assert bool((off <= 0).all()), "lse off by %g over its tolerance" % float(off.max())
        return o, tol, l, ltol


def _run(case, flags=0, **over):
    a = {**case.args(), **over}
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    ws[256:].view(torch.float32).fill_(3.0)    # what an earlier call may have left
    out, lse = fd.decode_attention_shared_prefix(workspace=ws, **a)
    assert fd.read_device_error(ws) == flags
    return out, lse


gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype,cache,d", [(BF, BF, 128), (BF, BF, 64), (F32, F32, 128),
                                           (F32, F32, 64), (BF, F8, 128)])
@pytest.mark.parametrize("page", [0, 8, 16, 64, 256])
def test_types_and_layouts(dtype, cache, d, page):
    c = Case(dtype, cache, d, groups=((5, 300),), own=(5, 0, 9, 33, 1), page=page, seed=page)
    c.check(*_run(c))
    c = Case(dtype, cache, d, groups=((3, 129), (1, 0), (2, 515)), own=(5, 0, 70), page=page,
             behind=2, seed=page + 1)
    c.check(*_run(c))


@gpu
@pytest.mark.parametrize("length", [1, 7, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_prompt_lengths(length):
    for cache in (BF, F8):
        c = Case(BF, cache, groups=((2, length),), own=(3, 0), cap=1024, seed=length)
        c.check(*_run(c))


@gpu
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 16, 64])
@pytest.mark.parametrize("cache", [BF, F8, F32])
def test_splits(splits, cache):
    c = Case(F32 if cache == F32 else BF, cache, groups=((3, 700), (2, 40)), own=(90, 0, 300), seed=splits)
    want = c.check(*_run(c, prefix_splits=splits, num_splits=splits))
    c.check(*_run(c, prefix_splits=splits, num_splits=1), want=want)


@gpu
@pytest.mark.parametrize("Hq,Hkv,Q", [(1, 1, 1), (8, 8, 1), (16, 2, 1), (16, 1, 1), (32, 1, 1), (64, 1, 1),
                                      (8, 2, 2), (8, 2, 4), (6, 3, 3), (4, 4, 16), (8, 1, 8)])
@pytest.mark.parametrize("rows", [1, 3, 17])
def test_heads_and_query_tokens(Hq, Hkv, Q, rows):
    c = Case(Hq=Hq, Hkv=Hkv, Q=Q, groups=((rows, 150),), own=(Q, Q + 3, 0, 1, 40), seed=rows)
    c.check(*_run(c))
    if Hq // Hkv * Q <= 32:
        c = Case(cache=F8, Hq=Hq, Hkv=Hkv, Q=Q, groups=((rows, 150),), own=(Q, Q + 3, 0, 1, 40), seed=rows)
        c.check(*_run(c))
    if Hq // Hkv * Q <= 16:
        c = Case(F32, Hq=Hq, Hkv=Hkv, Q=Q, groups=((rows, 150),), own=(Q, Q + 3, 0, 1, 40), seed=rows)
        c.check(*_run(c))


@gpu
@pytest.mark.parametrize("rows", [31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_row_tiles(rows):
    # 4 query rows each: the borders of tiles of 64, 128 and 256 query rows
    for cache in (BF, F8):
        c = Case(cache=cache, Hq=4, Hkv=1, groups=((rows, 270),), own=(4, 0, 11), seed=rows)
        c.check(*_run(c))
    c = Case(Hq=4, Hkv=1, groups=((rows, 140), (3, 270), (rows, 5)), own=(4, 0, 11), seed=rows)
    c.check(*_run(c))


@gpu
def test_many_groups():
    groups = tuple(((i * 5) % 3, (i * 37) % 200) for i in range(70))
    c = Case(Hq=4, Hkv=2, groups=groups, own=(3, 0, 17), behind=3, seed=4)
    c.check(*_run(c))


@gpu
@pytest.mark.parametrize("cache", [BF, F8, F32])
@pytest.mark.parametrize("rows", [1, 3, 64])
def test_one_group_and_rows_behind_it(cache, rows):
    c = Case(F32 if cache == F32 else BF, cache, groups=((rows, 150),), own=(5, 33, 1), behind=rows + 1, seed=rows)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    ws[256:].view(torch.float32).fill_(3.0)    # what an earlier call may have left
    c.check(*fd.decode_attention_shared_prefix(workspace=ws, **c.args()))


@gpu
def test_rows_without_any_key():
    c = Case(groups=((2, 0), (1, 30)), own=(0, 4, 0), behind=2, cap=64, seed=5)
    out, lse = _run(c)
    c.check(out, lse)
    for b in (0, 3):
        assert not out[b].any() and bool(torch.isneginf(lse[b]).all())


@gpu
@pytest.mark.parametrize("cache", [BF, F8, F32])
def test_large_scores(cache):
    # maxima that grow along the prompt and gaps of hundreds between keys
    c = Case(F32 if cache == F32 else BF, cache, groups=((4, 900),), own=(60, 3), scale=6.0, spikes=True, seed=6)
    c.check(*_run(c))
    c.check(*_run(c, prefix_splits=5))


@gpu
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_output_types_and_strides(out_dtype):
    c = Case(groups=((3, 100),), seed=7)
    out = torch.zeros(3, 8, 160, dtype=out_dtype, device="cuda")[:, :, 16:144]
    got, lse = _run(c, out=out)
    c.check(got, lse, out_dtype)
    c = Case(Q=2, groups=((3, 100),), own=(2, 9), seed=8)
    a = c.args()
    wide = torch.zeros(3, 2, 8, 256, dtype=BF, device="cuda")
    wide[..., 64:192] = a["q"]
    c.check(*_run(c, q=wide[..., 64:192]))


@gpu
def test_prompt_and_rows_laid_out_differently():
    for cache in (BF, F8):
        c = Case(cache=cache, groups=((2, 100), (2, 33)), own=(7, 30), page=16, own_page=0, seed=9)
        c.check(*_run(c))
        c = Case(cache=cache, groups=((2, 100), (2, 33)), own=(7, 30), page=0, own_page=32, seed=10)
        c.check(*_run(c))


@gpu
def test_strided_prefix():
    # heads outside the tokens: a [tokens, heads, d] cache seen as [1, heads, tokens, d]
    c = Case(groups=((3, 200),), seed=11)
    a = c.args()
    k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (a["k_prefix"], a["v_prefix"]))
    c.check(*_run(c, k_prefix=k, v_prefix=v))


@gpu
def test_paths_agree():
    c = Case(groups=((40, 300),), own=(5, 40), seed=12)
    want = c.check(*_run(c, options=fd.options(path=fd.FD_PATH_SIMT)))
    c.check(*_run(c, options=fd.options(path=fd.FD_PATH_MMA)), want=want)
    c.check(*_run(c), want=want)


@gpu
def test_same_result_every_time():
    for cache in (BF, F8, F32):
        c = Case(F32 if cache == F32 else BF, cache, groups=((70, 500), (3, 900)), own=(5, 40), seed=13)
        a = _run(c)
        for _ in range(3):
            b = _run(c)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_device_flags():
    c = Case(groups=((2, 60), (2, 40)), own=(4,), page=16, seed=14)
    a = c.args()
    table = a["prefix_table"].clone()
    table[0, 1] = 10000
    for name, value, flag in [("prefix_lens", _ints(60, 4000).cuda(), fd.FD_DEVFLAG_SEQ_LEN | fd.FD_DEVFLAG_PAGE),
                              ("prefix_lens", _ints(-1, 40).cuda(), fd.FD_DEVFLAG_SEQ_LEN),
                              ("group_start", _ints(0, 3, 2).cuda(), fd.FD_DEVFLAG_OFFSETS),
                              ("group_start", _ints(1, 2, 4).cuda(), fd.FD_DEVFLAG_OFFSETS),
                              ("group_start", _ints(0, 2, 9).cuda(), fd.FD_DEVFLAG_OFFSETS),
                              ("prefix_table", table, fd.FD_DEVFLAG_PAGE)]:
        for options in (None, fd.options(path=fd.FD_PATH_SIMT)):
            _run(c, flags=flag, options=options, **{name: value})
    # the tokens of a bad page are left out: row 0's prompt without tokens 16 .. 31
    d = Case(groups=((2, 60), (2, 40)), own=(4,), page=16, seed=14)
    keep = [t for t in range(60) if not 16 <= t < 32]
    d.kp[0, :, :44], d.vp[0, :, :44] = d.kp[0, :, keep], d.vp[0, :, keep]
    d.plens = [44, 40]
    for options in (None, fd.options(path=fd.FD_PATH_SIMT)):
        d.check(*_run(c, flags=fd.FD_DEVFLAG_PAGE, prefix_table=table, options=options))


@gpu
@pytest.mark.parametrize("cache", [BF, F8])
@pytest.mark.parametrize("rows,stall", [(3, 0), (3, 1), (3, 4), (90, 0), (90, 5)])
def test_stalled_copies_end_with_a_flag(cache, rows, stall):
    """Copies that never arrive: the waits run out, the call ends with a flag, rows that the
    stalled CTA (row tile 0, kv head 0, split 0) does not serve are right, and the same workspace
    then gives right results."""
    c = Case(cache=cache, groups=((rows, 900),), own=(5, 40), seed=17)
    a = c.args()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    out, lse = fd.decode_attention_shared_prefix(workspace=ws, selftest_stall=stall, prefix_splits=1, **a)
    assert fd.read_device_error(ws) == fd.FD_DEVFLAG_TIMEOUT
    got = fd.decode_attention_shared_prefix(workspace=ws, prefix_splits=1, **a)
    assert fd.read_device_error(ws) == 0
    c.check(*got)
    assert torch.equal(out[:, 4:], got[0][:, 4:]) and torch.equal(lse[:, 4:], got[1][:, 4:])


@gpu
def test_stall_past_the_last_copy_changes_nothing():
    c = Case(groups=((3, 300),), own=(5, 40), seed=18)
    a = c.args()
    want = _run(c)
    got = _run(c, selftest_stall=1000)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_two_threads_on_one_stream():
    """Two threads' calls, interleaved launch by launch on one stream, each with its own buffers."""
    import threading
    cases = [Case(groups=((3, 300),), own=(5, 40), seed=19),
             Case(cache=F8, groups=((70, 500), (2, 90)), own=(5, 40), seed=20)]
    args = [c.args() for c in cases]
    want = [_run(c) for c in cases]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        got = [fd.decode_attention_shared_prefix(workspace=ws, stream=stream, **args[i]) for _ in range(40)]
        stream.synchronize()
        if not all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not wrong


@gpu
def test_inputs_written_just_before_the_call():
    """Queries, lengths, own keys and prompts rewritten on the stream right before each call."""
    c = Case(groups=((20, 700), (30, 300)), own=(5, 40, 300), page=16, seed=21)
    a = c.args()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    want = fd.decode_attention_shared_prefix(workspace=ws, **a)
    names = ("q", "k_prefix", "v_prefix", "k_cache", "v_cache", "seq_lens", "prefix_lens",
             "group_start", "prefix_table", "block_table")
    kept = {n: a[n].clone() for n in names}
    for _ in range(30):
        for n in ("q", "k_cache", "v_cache", "k_prefix", "v_prefix"):
            a[n].fill_(3.0)
        a["seq_lens"].fill_(1)
        a["prefix_lens"].fill_(1)
        fd.decode_attention_shared_prefix(workspace=ws, **a)
        for n in names:
            a[n].copy_(kept[n])
        got = fd.decode_attention_shared_prefix(workspace=ws, **a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_tensors_elsewhere_are_refused():
    c = Case(groups=((3, 30),), own=(5,), seed=22)
    for name in ("q", "prefix_lens", "k_cache", "seq_lens"):
        a = c.args()
        a[name] = a[name].cpu()
        with pytest.raises(ValueError):
            fd.decode_attention_shared_prefix(**a)


@gpu
def test_streams_and_shared_workspace():
    c = Case(groups=((3, 300),), own=(5, 40), seed=15)
    a = c.args()
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    want = fd.decode_attention_shared_prefix(workspace=ws, **a)
    other = Case(groups=((9, 77), (1, 300)), own=(5, 40), seed=16)
    b = other.args()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):                          # calls of different sizes in one workspace
        got2 = fd.decode_attention_shared_prefix(workspace=ws, stream=s, **b)
        got = fd.decode_attention_shared_prefix(workspace=ws, stream=s, **a)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    other.check(*got2)


@gpu
@pytest.mark.parametrize("seed", range(40))
def test_random_draws(seed):
    """Random types, heads, groups, lengths, layouts and split counts."""
    import random
    r = random.Random(seed)
    cache = r.choice([BF, BF, F8, F32])
    Hkv = r.choice([1, 2, 3, 4])
    G = r.choice([1, 2, 4, 8])
    Q = r.choice([1, 1, 2, 3]) if G <= 4 else 1
    groups = tuple((r.choice([0, 1, 2, 7, 40]), r.choice([0, 1, 63, 128, 200, 333, 700]))
                   for _ in range(r.choice([1, 1, 2, 5])))
    if sum(n for n, _ in groups) == 0:
        groups = ((3, 150),)
    c = Case(F32 if cache == F32 else BF, cache, 128 if cache == F8 else r.choice([64, 128]), Hkv * G, Hkv, Q,
             groups, [r.choice([0, 1, 5, 33, 120]) for _ in range(6)], page=r.choice([0, 8, 16, 32, 128]),
             behind=r.choice([0, 0, 2]), cap=704, seed=seed)
    c.check(*_run(c, prefix_splits=r.choice([0, 0, 1, 3]), num_splits=r.choice([0, 0, 2])))


@gpu
@pytest.mark.parametrize("cache", [BF, F8])
def test_serving_loop(cache):
    """A batch on two prompts decodes in a captured graph: each step appends the rotated keys
    and values of one token a row (its cache continues its prompt), then attends; every step's
    output equals plain attention over the whole sequence, evaluated in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, Hq, Hkv, d, page, steps = 5, 8, 2, 128, 16, 20
    plens, sizes = [150, 37], [3, 2]
    group = [0, 0, 0, 1, 1]
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    scale = torch.tensor([0.02, 0.03], device="cuda") if cache == F8 else None
    pages = 64
    kc, vc = (torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(F8) if cache == F8
              else torch.zeros(pages, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    pt = order[:20].view(2, 10).contiguous()
    bt = order[20:20 + B * 2].view(B, 2).contiguous()
    cs = fd.rope_table(256, d, device="cuda")
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    kp, vp = rnd(sum(plens), Hkv, d), rnd(sum(plens), Hkv, d)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    fd.append_kv(None, kp, vp, kc, vc, ints(*plens), cs, cu_tokens=ints(0, plens[0], sum(plens)),
                 block_table=pt, page_size=page, k_scale=scale, v_scale=scale, workspace=ws)
    q, k, v = rnd(B, Hq, d), rnd(B, Hkv, d), rnd(B, Hkv, d)
    lens, offs = torch.zeros(B, dtype=torch.int32, device="cuda"), ints(*[plens[i] for i in group])
    start, pl = ints(0, 3, 5), ints(*plens)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(B, Hq, device="cuda")

    def step():
        lens.add_(1)
        fd.append_kv(q, k, v, kc, vc, lens, cs, pos_offset=offs, block_table=bt, page_size=page,
                     k_scale=scale, v_scale=scale, q_out=qr, workspace=ws)
        fd.decode_attention_shared_prefix(qr, kc, vc, pl, kc, vc, lens, group_start=start,
                                          prefix_table=pt, block_table=bt, page_size=page,
                                          k_scale=scale, v_scale=scale, out=out, lse_out=lse, workspace=ws)

    step()                                      # warm up, then start over
    lens.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    lens.zero_()

    def turned(x, pos):                         # x [H, d], rotated in 64 bits and rounded once
        c, s = cs[pos, :d // 2].double(), cs[pos, d // 2:].double()
        a, b = x[:, :d // 2].double(), x[:, d // 2:].double()
        return torch.cat([a * c - b * s, b * c + a * s], 1)

    def stored(x):                              # what the cache holds of it
        if cache != F8:
            return x.to(BF).double()
        return ((x / scale.double()[:, None]).clamp(-448, 448).float().to(F8).double() * scale.double()[:, None])

    first = [0, plens[0]]
    hist = [[(stored(turned(kp[first[p] + t], t)), stored(vp[first[p] + t].double())) for t in range(plens[p])]
            for p in range(2)]
    mine = [[] for _ in range(B)]
    step_of = 2.0 ** -4 if cache == F8 else 2.0 ** -8   # a code next to a border may fall to either side
    for n in range(steps):
        q.copy_(rnd(B, Hq, d)), k.copy_(rnd(B, Hkv, d)), v.copy_(rnd(B, Hkv, d))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            pos = plens[group[b]] + n
            mine[b].append((stored(turned(k[b], pos)), stored(v[b].double())))
            keys = hist[group[b]] + mine[b]
            kk, vv = torch.stack([x for x, _ in keys], 1), torch.stack([y for _, y in keys], 1)
            x = turned(q[b], pos).to(BF).double().view(Hkv, Hq // Hkv, d)
            s = x @ kk.transpose(1, 2) / math.sqrt(d)
            l = torch.logsumexp(s, -1)
            w = (s - l[..., None]).exp()
            o = w @ vv
            # few elements sit that near a border: one step of one key moves a score by at
            # most step_of * max |q_i k_i| / sqrt(d)
            ds = step_of * float(x.abs().max() * kk.abs().max()) / math.sqrt(d)
            A = w @ vv.abs()
            assert bool(((out[b].double().view_as(o) - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * ds + 1e-3) * A).all())
            assert bool(((lse[b].double().view_as(l) - l).abs() <= ds + 1e-3).all())
    assert fd.read_device_error(ws) == 0
