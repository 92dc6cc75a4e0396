"""fd_append_kv: new tokens' keys and values written into the cache, rotated by position.

GPU results are compared with the definition evaluated in 64 bits.  Tolerances: a value is
rounded once to its type, off by at most half a step (bf16 2^-8, f32 2^-24 relative; e4m3
2^-4 relative or 2^-10 below its normal range), after two products and a sum in f32, off by
at most 3 * 2^-24 (|x_a| + |x_b|).  v is copied: equal bit for bit.  Slots that no token
writes keep their bytes.
"""
import pytest
import torch

fd = pytest.importorskip("decode_attention_05_gb300")

INVALID, UNSUPPORTED = 1, 2
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


# ------------------------------------------------------------------ refusals (no GPU)


def _cpu_case(**over):
    a = dict(q=torch.zeros(3, 4, 128, dtype=torch.bfloat16),
             k=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
             v=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
             k_cache=torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16),
             v_cache=torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16),
             seq_lens=torch.ones(3, dtype=torch.int32), cos_sin=torch.zeros(16, 128), stream=0)
    a.update(over)
    return a


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


REFUSED = [
    ("v heads", dict(v=_bf(3, 1, 128)), INVALID),
    ("v dtype", dict(v=torch.zeros(3, 2, 128)), INVALID),
    ("q tokens", dict(q=_bf(2, 4, 128)), INVALID),
    ("q head dim", dict(q=_bf(3, 4, 64)), INVALID),
    ("q_out shape", dict(q_out=_bf(3, 3, 128)), INVALID),
    ("q_out without q", dict(q=None, q_out=_bf(3, 4, 128)), INVALID),
    ("q_out overlapping rows", dict(q_out=_bf(1, 4, 128).expand(3, 4, 128)), INVALID),
    ("tokens differ from rows", dict(k=_bf(2, 2, 128), v=_bf(2, 2, 128), q=None), INVALID),
    ("cache heads", dict(k_cache=_bf(3, 1, 16, 128), v_cache=_bf(3, 1, 16, 128)), INVALID),
    ("cache shapes", dict(v_cache=_bf(3, 2, 8, 128)), INVALID),
    ("cache dtype", dict(k_cache=torch.zeros(3, 2, 16, 128), v_cache=torch.zeros(3, 2, 16, 128)),
     UNSUPPORTED),
    ("cache dtypes differ", dict(v_cache=torch.zeros(3, 2, 16, 128)), INVALID),
    ("fp8 from f32", dict(q=None, k=torch.zeros(3, 2, 128), v=torch.zeros(3, 2, 128),
                          k_cache=_f8(3, 2, 16, 128), v_cache=_f8(3, 2, 16, 128)), UNSUPPORTED),
    ("fp8 head dim 64", dict(q=None, k=_bf(3, 2, 64), v=_bf(3, 2, 64), cos_sin=None,
                             k_cache=_f8(3, 2, 16, 64), v_cache=_f8(3, 2, 16, 64)), UNSUPPORTED),
    ("scales without fp8", dict(k_scale=torch.ones(2)), INVALID),
    ("head dim", dict(q=None, k=_bf(3, 2, 96), v=_bf(3, 2, 96), cos_sin=None,
                      k_cache=_bf(3, 2, 16, 96), v_cache=_bf(3, 2, 16, 96)), UNSUPPORTED),
    ("page size without table", dict(page_size=16), INVALID),
    ("page size", dict(page_size=12, block_table=torch.zeros(3, 4, dtype=torch.int32)), INVALID),
    ("page size of the pool", dict(page_size=32, block_table=torch.zeros(3, 4, dtype=torch.int32)),
     INVALID),
    ("table dtype", dict(page_size=16, block_table=torch.zeros(3, 4)), INVALID),
    ("rotated dims", dict(cos_sin=torch.zeros(16, 24)), UNSUPPORTED),
    ("more rotated dims than d", dict(cos_sin=torch.zeros(16, 144)), INVALID),
    ("table of angles 3-D", dict(cos_sin=torch.zeros(1, 16, 128)), INVALID),
    ("rope style", dict(rope_style=2), INVALID),
    ("pos_offset without rotation", dict(cos_sin=None, pos_offset=torch.zeros(3, dtype=torch.int32)),
     INVALID),
    ("misaligned k", dict(k=_bf(3 * 2 * 128 + 8)[1:-7].view(3, 2, 128)), INVALID),
    ("k strides", dict(q=None, k=_bf(3 * 260).as_strided((3, 2, 128), (260, 130, 1))), INVALID),
    ("overlapping cache rows", dict(k_cache=_bf(3, 2, 16, 128).as_strided((3, 2, 16, 128), (4096, 2048, 64, 1))),
     INVALID),
]


@pytest.mark.parametrize("name,over,status", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(name, over, status):
    with pytest.raises(fd.FdError) as e:
        fd.append_kv(**_cpu_case(**over))
    assert e.value.status == status


def test_binding_checks_host_visible_sizes():
    for over in (dict(seq_lens=torch.ones(2, dtype=torch.int32)),
                 dict(cu_tokens=torch.zeros(3, dtype=torch.int32)),
                 dict(pos_offset=torch.zeros(4, dtype=torch.int32)),
                 dict(k_cache=_f8(3, 2, 16, 128), v_cache=_f8(3, 2, 16, 128), k_scale=torch.ones(1))):
        with pytest.raises(ValueError):
            fd.append_kv(**_cpu_case(**over))
    with pytest.raises(TypeError):
        fd.append_kv(**_cpu_case(seq_lens=torch.ones(3, dtype=torch.int64)))


def test_rope_table():
    t = fd.rope_table(100, 32, base=500.0)
    assert t.shape == (100, 32) and t.dtype == torch.float32
    r, i = 77, 5
    angle = torch.tensor(float(r), dtype=torch.float64) * 500.0 ** (-2 * i / 32)
    assert abs(float(t[r, i]) - float(angle.cos())) <= 2.0 ** -24
    assert abs(float(t[r, 16 + i]) - float(angle.sin())) <= 2.0 ** -24


# ------------------------------------------------------------------ the definition, 64 bits


def _rotated(x, pos, cos_sin, style):
    """x [H, d] in f64 at rotary position pos; also |x_a| + |x_b| of every dim's pair."""
    y, mag = x.clone(), x.abs()
    if cos_sin is None:
        return y, mag
    h = cos_sin.shape[1] // 2
    c, s = cos_sin[pos, :h].double(), cos_sin[pos, h:].double()
    i = torch.arange(h)
    a, b = (i, i + h) if style == fd.FD_ROPE_HALF else (2 * i, 2 * i + 1)
    y[:, a] = x[:, a] * c - x[:, b] * s
    y[:, b] = x[:, b] * c + x[:, a] * s
    mag[:, a] = mag[:, b] = x[:, a].abs() + x[:, b].abs()
    return y, mag


def _check_close(got, want, mag, dtype, scale=None):
    if dtype == torch.float8_e4m3fn:
        want, mag = want / scale, mag / scale
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        want = want.clamp(-448, 448)
        tol = (2.0 ** -4 * want.abs()).clamp(min=2.0 ** -10) + 2.0 ** -22 * mag
        ok = (got - want).abs() <= tol
        assert bool((ok | nan).all())
        return
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    fine = ~nan & ~inf
    tol = HALF_STEP[dtype] * want.abs() + 3 * 2.0 ** -24 * mag
    assert bool(((got - want).abs()[fine] <= tol[fine]).all())


def _run_case(dtype, cache, d, Hq, Hkv, lens, new, page, rot, style, multi=False, offsets=None,
              with_q=True, in_place=False, pad=0, seed=0, special=False):
    """One call against the definition; `new`: tokens of each row, `pad` more behind them."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(lens), sum(new) + pad
    ragged = not multi and (pad or any(n != 1 for n in new))
    qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(dtype)
    if special:
        qkv[0, ::7] = float("inf")
        qkv[-1, ::5] = float("nan")
        qkv[T // 2] = 3e4
    dev = qkv.cuda()
    cut = lambda x: (x[:, :Hq * d].unflatten(1, (Hq, d)),  # noqa: E731
                     x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)),
                     x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)))
    q, k, v = cut(dev)
    hq, hk, hv = (x.double() for x in cut(qkv))
    if multi:
        q, k, v = (x.unflatten(0, (B, new[0])) for x in (q, k, v))
    cap = max(max(lens), 1)
    table = None
    if page:
        width = -(-cap // page)
        pages = B * width + 3
        table = torch.randperm(pages, generator=g)[:B * width].view(B, width).to(torch.int32)
        shape = (pages, Hkv, page, d)
    else:
        shape = (B, Hkv, cap, d)
    fill = lambda: torch.randn(shape, generator=g).to(torch.bfloat16).to(cache)  # noqa: E731
    k0, v0 = fill(), fill()
    kc, vc = k0.cuda(), v0.cuda()
    ks = vs = None
    if cache == torch.float8_e4m3fn:
        ks, vs = torch.rand(Hkv, generator=g) * 0.02 + 0.004, torch.rand(Hkv, generator=g) * 0.02 + 0.004
    offs = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    most = cap + (max(offsets) if offsets else 0)
    cos_sin = fd.rope_table(most, rot) if rot else None
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
    q_out = None
    if with_q:
        q_out = q if in_place else torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    got = fd.append_kv(q if with_q else None, k, v, kc, vc,
                       torch.tensor(lens, dtype=torch.int32).cuda(), gpu(cos_sin),
                       rope_style=style, pos_offset=gpu(offs),
                       cu_tokens=torch.tensor(cu, dtype=torch.int32).cuda() if ragged else None,
                       block_table=gpu(table), page_size=page, k_scale=gpu(ks), v_scale=gpu(vs),
                       q_out=q_out, workspace=ws)
    assert fd.read_device_error(ws) == 0
    if with_q:
        got = got.reshape(T, Hq, d).cpu()
        before = torch.full((T, Hq, d), 7.0, dtype=dtype) if not in_place else cut(qkv)[0]
    kc, vc = kc.cpu(), vc.cpu()
    touched = torch.zeros(shape[0], shape[2], dtype=torch.bool)
    for b in range(B):
        for i in range(new[b]):
            t, pos = cu[b] + i, lens[b] - new[b] + i
            if pos < 0:
                if with_q:
                    assert torch.equal(got[t], before[t])
                continue
            rp = pos + (offsets[b] if offsets else 0)
            place, slot = (int(table[b, pos // page]), pos % page) if page else (b, pos)
            touched[place, slot] = True
            want, mag = _rotated(hk[t], rp, cos_sin, style)
            scale = None if ks is None else ks.double()[:, None]
            _check_close(kc[place, :, slot].double(), want, mag, cache, scale)
            scale = None if vs is None else vs.double()[:, None]
            if cache == torch.float8_e4m3fn:
                _check_close(vc[place, :, slot].double(), hv[t], torch.zeros_like(hv[t]), cache, scale)
            else:
                assert torch.equal(vc[place, :, slot].nan_to_num(9.0), hv[t].to(cache).nan_to_num(9.0))
            if with_q:
                want, mag = _rotated(hq[t], rp, cos_sin, style)
                _check_close(got[t].double(), want, mag, dtype)
    if with_q and pad:
        assert torch.equal(got[sum(new):], before[sum(new):])
    raw = torch.uint8 if cache == torch.float8_e4m3fn else torch.int16 if cache == torch.bfloat16 else torch.int32
    for now, was in ((kc, k0), (vc, v0)):
        now, was = now.view(raw).transpose(1, 2), was.view(raw).transpose(1, 2)
        assert torch.equal(now[~touched], was[~touched])


BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H, I = fd.FD_ROPE_HALF, fd.FD_ROPE_INTERLEAVED


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache,d", [(BF, BF, 128), (BF, BF, 64), (F32, F32, 128),
                                           (F32, F32, 64), (BF, F8, 128)])
@pytest.mark.parametrize("page", [0, 8, 16, 64])
@pytest.mark.parametrize("style", [H, I])
def test_types_and_layouts(dtype, cache, d, page, style):
    _run_case(dtype, cache, d, 8, 2, [1, 16, 17, 40, 33], [1] * 5, page, d, style, seed=page)
    _run_case(dtype, cache, d, 4, 4, [5, 16, 31, 0, 64], [5, 0, 17, 0, 40], page, d, style, seed=1 + page)
    _run_case(dtype, cache, d, 3, 1, [3, 4, 70], [3] * 3, page, d, style, multi=True, seed=2 + page)


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 112, 128])
@pytest.mark.parametrize("style", [H, I])
def test_rotated_dims(rot, style):
    _run_case(BF, BF, 128, 4, 2, [9, 30], [4, 7], 16, rot, style, seed=rot)
    if rot <= 64:
        _run_case(F32, F32, 64, 4, 2, [9, 30], [4, 7], 0, rot, style, seed=rot)


@pytest.mark.gpu
def test_one_token_one_row_and_odd_heads():
    _run_case(BF, BF, 128, 1, 1, [1], [1], 0, 128, H)
    _run_case(BF, BF, 64, 7, 3, [2, 9], [1, 1], 8, 64, I)
    _run_case(F32, F32, 128, 1, 1, [100], [100], 16, 128, H)


@pytest.mark.gpu
def test_without_q_and_in_place():
    _run_case(BF, BF, 128, 4, 2, [9, 30], [4, 7], 16, 128, H, with_q=False)
    for style in (H, I):
        _run_case(BF, BF, 128, 4, 2, [9, 30], [4, 7], 16, 128, style, in_place=True)


@pytest.mark.gpu
def test_padding_rows_and_offsets():
    # rows shorter than their new tokens, empty rows, tokens behind the last row
    _run_case(BF, BF, 128, 4, 2, [0, 2, 5, 0], [1, 4, 5, 3], 16, 128, H, pad=9)
    _run_case(BF, BF, 128, 4, 2, [0, 1, 0], [1, 1, 1], 0, 128, H)
    _run_case(BF, BF, 128, 4, 2, [3, 1, 20], [1, 1, 1], 16, 64, H, offsets=[1000, 0, 131])


@pytest.mark.gpu
def test_special_values():
    for cache in (BF, F8):
        _run_case(BF, cache, 128, 4, 2, [9, 30], [4, 7], 16, 0, H, special=True)
    _run_case(F32, F32, 64, 4, 2, [9, 30], [4, 7], 0, 0, H, special=True)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 31, 32, 33, 500, 1100])
def test_many_rows_are_found(B):
    new = [(i * 7) % 4 for i in range(B)]
    new[-1] += 1
    _run_case(BF, BF, 64, 2, 1, [n + i % 5 for i, n in enumerate(new)], new, 8, 64, H, seed=B)


@pytest.mark.gpu
def test_large_enough_for_several_rows_a_warp():
    # past the size where a warp takes four row groups at a time
    _run_case(BF, BF, 128, 28, 4, [700, 300], [640, 300], 16, 128, H, pad=5)
    _run_case(F32, F32, 64, 21, 5, [900, 300], [840, 300], 0, 32, I)


@pytest.mark.gpu
def test_device_flags():
    mk = lambda **o: {k: (x.cuda() if isinstance(x, torch.Tensor) else x)  # noqa: E731
                      for k, x in _cpu_case(q=None, stream=None, **o).items()}
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    ones = torch.ones(3, 2, 128, dtype=torch.bfloat16)
    for over, flag, written in [
            (dict(seq_lens=ints(17, 1, -1)), fd.FD_DEVFLAG_SEQ_LEN, [1]),
            (dict(cos_sin=torch.zeros(4, 128), seq_lens=ints(4, 5, 1)), fd.FD_DEVFLAG_POSITION, [0, 2]),
            (dict(pos_offset=ints(0, -5, 16)), fd.FD_DEVFLAG_POSITION, [0]),
            (dict(cu_tokens=ints(0, 1, 0, 3)), fd.FD_DEVFLAG_OFFSETS, None),
            (dict(cu_tokens=ints(1, 2, 3, 3)), fd.FD_DEVFLAG_OFFSETS, [0, 1]),
            (dict(page_size=16, block_table=ints(0, 3, -1).view(3, 1)), fd.FD_DEVFLAG_PAGE, [0])]:
        a = mk(k=ones, v=ones, **over)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        fd.append_kv(workspace=ws, **a)
        assert fd.read_device_error(ws) == flag
        if written is not None:
            rows = a["v_cache"].float().abs().amax((1, 2, 3)).cpu()
            assert [b for b in range(3) if rows[b] > 0] == written
        fd.append_kv(**a)                      # the same without a place for flags
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A slot whose element offset needs more than 32 bits (4.4 billion elements into the cache)."""
    shape = (1, 2, 1 << 24, 128)
    kc = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    vc = kc.as_strided(shape, kc.stride())
    n = (1 << 24) - 3
    kc[0, 1, n - 1:n + 1] = 5.0
    k = torch.full((1, 2, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    fd.append_kv(None, k, k, kc, vc, torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert float(kc[0, 1, n - 1].float().sum()) == 256.0
    assert float(kc[0, 1, n].float().sum()) == 640.0


@pytest.mark.gpu
def test_tensors_elsewhere_are_refused():
    for name in ("q", "k_cache", "seq_lens"):
        a = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in _cpu_case().items()}
        a[name] = a[name].cpu()
        with pytest.raises(ValueError):
            fd.append_kv(**a)
    with pytest.raises(ValueError):
        fd.append_kv(**_cpu_case())


@pytest.mark.gpu
def test_other_stream_and_graph():
    d, ws = 128, torch.zeros(256, dtype=torch.uint8, device="cuda")
    k = torch.randn(4, 2, d, device="cuda").to(BF)
    q = torch.randn(4, 8, d, device="cuda").to(BF)
    kc, vc = (torch.zeros(4, 2, 32, d, device="cuda", dtype=BF) for _ in range(2))
    lens = torch.tensor([3, 9, 1, 20], dtype=torch.int32, device="cuda")
    cs = fd.rope_table(32, d, device="cuda")
    want_q = fd.append_kv(q, k, k, kc, vc, lens, cs, workspace=ws)
    want = kc.clone(), vc.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kc.zero_(), vc.zero_()
    torch.cuda.synchronize()
    got = fd.append_kv(q, k, k, kc, vc, lens, cs, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(got, want_q) and torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.append_kv(q, k, k, kc, vc, lens, cs, q_out=out, workspace=ws)
    kc.zero_(), vc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_q) and torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    lens += 1                                  # the next step writes the next slots
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(vc[1, :, 8], vc[1, :, 9]) and not torch.equal(kc[1, :, 8], kc[1, :, 9])
