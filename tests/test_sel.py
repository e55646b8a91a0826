"""The per-channel selective scan, its one-token step and its conv, against a
64-bit recurrence on the same inputs.

Bounds, relative to the sum of the absolute values of what is added (`size`):
an exponential has a relative error of 2^-22 (the special-function unit) and of
|dt A| times the errors of dt, A and their product, under 2^-20 in all for the
decays that still matter (|dt A| < 4, beyond it what is kept is 2% of what is
added). A state that remembers m tokens adds up m of the former, which is what
STEP times the longest length bounds; the sums over states and the skip are
within 1e-5 of the size. bf16 outputs are rounded once, by at most 2^-8.
"""

import ctypes

import pytest
import torch

import mamba_recurrent_state_b200 as m2

F32, BF16 = m2.M2_F32, m2.M2_BF16
TYPES = {F32: torch.float32, BF16: torch.bfloat16}
BASE, STEP = 1e-5, 2.0 ** -22


class Layer:
    def __init__(self, shape, T, seed=1, z=True, groups_flat=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        act = TYPES[shape.act_dtype]
        draw = lambda *s, std=1.0, dt=act: torch.empty(s, dtype=dt, device="cuda").normal_(0, std, generator=g)  # noqa: E731
        uni = lambda *s, lo, hi: torch.empty(s, device="cuda").uniform_(lo, hi, generator=g)  # noqa: E731
        D, N, G = shape.D, shape.N, shape.G
        self.shape = shape
        self.params = m2.SelParams(uni(D, N, lo=1, hi=16).log(), uni(D, lo=1e-3, hi=0.1).expm1().log(), draw(D, dt=torch.float32))
        self.taps = m2.ConvParams(draw(D, shape.K, std=0.5), draw(D, std=0.1), 1)
        self.x, self.dt = draw(T, D), draw(T, D)
        self.B, self.C = draw(T, G, N), draw(T, G, N)
        self.z = draw(T, D) if z else None

    def reference(self, h, rows):
        """(y, final state, sizes) of consecutive token rows from state h [D, N], in 64 bits."""
        sh = self.shape
        rep = sh.D // sh.G
        A = -self.params.A_log.double().exp()
        skip, bias = self.params.D.double(), self.params.dt_bias.double()
        h, size = h.double(), h.double().abs()
        ys, ysizes = [], []
        for t in rows:
            x = self.x[t].double()
            dt = torch.nn.functional.softplus(self.dt[t].double() + bias, threshold=40)
            B, C = (v[t].double().repeat_interleave(rep, 0) for v in (self.B, self.C))
            decay = torch.exp(dt[:, None] * A)
            fresh = (dt * x)[:, None] * B
            h, size = h * decay + fresh, size * decay + fresh.abs()
            y, ysize = (h * C).sum(-1) + skip * x, (size * C.abs()).sum(-1) + (skip * x).abs()
            if self.z is not None:
                gate = self.z[t].double()
                gate = gate * torch.sigmoid(gate)
                y, ysize = y * gate, ysize * gate.abs()
            ys.append(y)
            ysizes.append(ysize)
        if not ys:
            return torch.zeros(0, sh.D, device="cuda").double(), h, torch.zeros(0, sh.D, device="cuda").double(), size
        return torch.stack(ys), h, torch.stack(ysizes), size


def within(got, want, size, length, dtype, what):
    bound = (BASE + STEP * length) * size
    if dtype == BF16:
        bound = bound + 2.0 ** -8 * want.abs()
    worst = ((got.double() - want).abs() - bound).max()
    assert worst <= 0, f"{what}: off by {worst:.3g} more than its bound"


def cache_of(shape, slots, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = m2.SelCache(shape, slots)
    c.ssm.normal_(0, 0.1, generator=g)
    c.conv.normal_(0, 1, generator=g)
    return c


def offsets(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_scan(layer, cache, lengths, slots, init, y, before, padding=()):
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    touched = set()
    for i, n in enumerate(lengths):
        rows = range(cu[i], cu[i + 1])
        s = int(slots[i])
        if s < 0 or i in padding:
            assert (y[cu[i]:cu[i + 1]] == 0).all()
            continue
        if n == 0:
            continue
        touched.add(s)
        h0 = before[s] if init is not None and init[i] else torch.zeros_like(before[s])
        ref, h, ysize, hsize = layer.reference(h0, rows)
        within(y[cu[i]:cu[i + 1]], ref, ysize, n, layer.shape.act_dtype, f"y of sequence {i}")
        within(cache.ssm[s], h, hsize, n, layer.shape.state_dtype, f"state of sequence {i}")
    for s in set(range(cache.num_slots)) - touched:
        assert torch.equal(cache.ssm[s], before[s])


# ---- host: refusals --------------------------------------------------------------

def test_shapes_and_sizes_on_the_host():
    L = m2.lib()
    for shape, want in ((m2.SelShape(8192, 16), m2.M2_OK), (m2.SelShape(40, 8, 5, 2, BF16, BF16), m2.M2_OK),
                        (m2.SelShape(12, 128, 3, 8, F32, F32), m2.M2_OK), (m2.SelShape(12, 16), m2.M2_ERR_UNSUPPORTED),
                        (m2.SelShape(64, 24), m2.M2_ERR_UNSUPPORTED), (m2.SelShape(64, 16, 3), m2.M2_ERR_INVALID_ARG),
                        (m2.SelShape(64, 16, 1, 1), m2.M2_ERR_UNSUPPORTED), (m2.SelShape(0, 16), m2.M2_ERR_INVALID_ARG),
                        (m2.SelShape(64, 16, 1, 4, m2.M2_F16), m2.M2_ERR_INVALID_ARG), (m2.SelShape(2**20, 8, 2**17), m2.M2_ERR_UNSUPPORTED)):
        assert m2.sel_shape_check(shape) == want, shape
    s = m2.SelShape(1000, 16, 1, 4, F32, BF16).c()
    a, b = ctypes.c_int64(), ctypes.c_int64()
    assert L.m2_sel_cache_bytes(ctypes.byref(s), 3, ctypes.byref(a), ctypes.byref(b)) == m2.M2_OK
    assert (a.value, b.value) == (3 * 64000, 3 * 6000)
    out = m2.m2_sel_cache()
    assert L.m2_sel_cache_wrap(ctypes.byref(s), 3, 0x1004, 0x2000, None, ctypes.byref(out)) == m2.M2_ERR_INVALID_ARG
    assert L.m2_sel_cache_wrap(ctypes.byref(s), 3, 0x1000, 0x2000, None, None) == m2.M2_ERR_INVALID_ARG


def test_entry_points_refuse_bad_arguments():
    L = m2.lib()
    s = m2.SelShape(64, 16, 2, 4, F32, BF16).c()
    cache = m2.m2_sel_cache()
    assert L.m2_sel_cache_wrap(ctypes.byref(s), 4, 0x100000, 0x200000, None, ctypes.byref(cache)) == m2.M2_OK
    c = ctypes.byref(cache)
    p = m2.m2_sel_params(0x300000, 0x300100, 0x300200)
    buf = 0x400000
    rows = dict(x=buf, xs=64, dt=buf, ds=64, B=buf, bs=32, C=buf, cs=32, z=buf, zs=64, y=buf, ys=64, idx=buf)
    bad = [dict(x=None), dict(xs=63), dict(xs=60), dict(dt=buf + 2), dict(ds=65), dict(B=None), dict(bs=31), dict(C=buf + 8),
           dict(cs=36), dict(z=buf + 4), dict(zs=8), dict(y=None), dict(ys=68), dict(idx=None)]
    for change in bad:
        v = list({**rows, **change}.values())
        assert L.m2_sel_state_update(c, ctypes.byref(p), 2, *v, None) == m2.M2_ERR_INVALID_ARG, change
        assert L.m2_sel_scan(c, ctypes.byref(p), 1, buf, 5, 5, *v, None, None) == m2.M2_ERR_INVALID_ARG, change
    v = list(rows.values())
    assert L.m2_sel_state_update(c, None, 2, *v, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_sel_state_update(c, ctypes.byref(p), -1, *v, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_sel_state_update(c, ctypes.byref(p), 0, *v, None) == m2.M2_OK
    assert L.m2_sel_state_update(c, ctypes.byref(p), 65536, *v, None) == m2.M2_ERR_UNSUPPORTED
    assert L.m2_sel_scan(c, ctypes.byref(p), 1, None, 5, 5, *v, None, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_sel_scan(c, ctypes.byref(p), 1, buf, 2**31, 5, *v, None, None) == m2.M2_ERR_UNSUPPORTED
    assert L.m2_sel_scan(c, ctypes.byref(p), 0, None, 0, 0, *v, None, None) == m2.M2_OK
    odd = m2.m2_sel_params(0x300004, 0x300100, 0x300200)
    assert L.m2_sel_state_update(c, ctypes.byref(odd), 2, *v, None) == m2.M2_ERR_INVALID_ARG
    taps = m2.m2_conv_params(0x500000, None, 1)
    conv = lambda **k: L.m2_sel_conv1d_update_varlen(c, ctypes.byref(taps), *{**dict(n=1, cu=buf, total=5, most=5, x=buf, xs=64, o=buf,  # noqa: E731
                                                                                   t=BF16, os=64, idx=buf, st=None), **k}.values())
    for change in (dict(cu=None), dict(x=None), dict(xs=60), dict(t=9), dict(os=63), dict(idx=None), dict(n=-1)):
        assert conv(**change) == m2.M2_ERR_INVALID_ARG, change
    assert conv(total=2**31) == m2.M2_ERR_UNSUPPORTED and conv(n=0, total=0) == m2.M2_OK


def test_binding_refuses_bad_tensors():
    shape = m2.SelShape(32, 16, 2)
    cache = m2.SelCache(shape, 4, device="cpu")
    params = m2.SelParams(torch.zeros(32, 16), torch.zeros(32), torch.zeros(32))
    x, B = torch.zeros(3, 32, dtype=torch.bfloat16), torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    ok = dict(x=x, dt=x, B=B, C=B, slot_idx=slots)
    for change in (dict(x=x.float()), dict(dt=x[:2]), dict(B=B[:, :1]), dict(C=B.transpose(1, 2)), dict(slot_idx=slots.long()),
                   dict(z=x[:, :16])):
        with pytest.raises(ValueError):
            m2.sel_state_update(cache, params, **{**ok, **change})
    with pytest.raises(ValueError, match="A_log"):
        m2.sel_state_update(cache, m2.SelParams(torch.zeros(32, 8), params.dt_bias, params.D), **ok)
    with pytest.raises(ValueError, match="CUDA device"):
        m2.sel_state_update(cache, params, **ok)
    with pytest.raises(ValueError):
        m2.sel_scan(cache, params, x, x, B, B, torch.tensor([0, 3]), slots[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        m2.sel_scan(cache, params, x, x, B, B, torch.tensor([0, 3], dtype=torch.int32), slots[:1])
    with pytest.raises(ValueError):
        m2.SelCache(shape, 4, ssm=torch.zeros(4, 32, 8))


# ---- prompts ---------------------------------------------------------------------

SHAPES = [m2.SelShape(64, 16, 1, 4, F32, BF16), m2.SelShape(136, 16, 1, 4, BF16, BF16), m2.SelShape(40, 8, 5, 4, F32, F32),
          m2.SelShape(520, 16, 1, 4, F32, F32), m2.SelShape(72, 32, 3, 4, BF16, F32), m2.SelShape(48, 64, 2, 4, F32, BF16),
          m2.SelShape(24, 128, 1, 4, BF16, BF16), m2.SelShape(12, 128, 3, 4, F32, F32), m2.SelShape(8, 16, 1, 4, F32, BF16)]


@pytest.mark.gpu
@pytest.mark.parametrize("z", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scan_of_packed_prompts(shape, z):
    lengths = [1, 0, 33, 64, 7, 130, 2]
    layer = Layer(shape, sum(lengths), z=z)
    cache = cache_of(shape, 9)
    slots = ints(4, 2, 0, -1, 8, 3, 6)
    init = torch.tensor([1, 1, 0, 1, 1, 1, 0], dtype=torch.uint8, device="cuda")
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets(lengths), slots, max_seqlen=130, z=layer.z,
                    has_initial_state=init)
    check_scan(layer, cache, lengths, slots, init, y, before)
    assert cache.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[1], [3], [31], [32], [129], [700], [5, 600], [1] * 40, [17] * 12], ids=lambda v: f"{len(v)}x{v[-1]}")
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_scan_lengths(lengths, act):
    shape = m2.SelShape(200, 16, 1, 4, F32, act)
    layer = Layer(shape, sum(lengths))
    cache = cache_of(shape, 64)
    slots = torch.randperm(64, device="cuda")[: len(lengths)].to(torch.int32)
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets(lengths), slots, max_seqlen=1, z=layer.z)
    check_scan(layer, cache, lengths, slots, None, y, before)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [m2.SelShape(64, 16, 1, 4, F32, BF16), m2.SelShape(40, 8, 1, 4, F32, F32), m2.SelShape(48, 32, 2, 4, BF16, BF16),
                                   m2.SelShape(24, 64, 1, 4, F32, F32), m2.SelShape(16, 128, 2, 4, F32, BF16)], ids=str)
def test_scan_in_segments(shape):
    """One long prompt of few channels is cut into segments; beside it an empty
    one, ones shorter than a segment or a tile, a padding row and a bad slot."""
    lengths = [1200, 0, 3, 65, 300, 1, 20, 9]
    layer = Layer(shape, sum(lengths))
    cache = cache_of(shape, 9)
    slots = ints(4, 2, 0, 1, 8, 3, -1, 9)
    init = torch.tensor([1, 1, 0, 1, 1, 1, 0, 1], dtype=torch.uint8, device="cuda")
    before = cache.ssm.clone()
    y = torch.full((sum(lengths), shape.D), 9.0, dtype=TYPES[shape.act_dtype], device="cuda")
    m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets(lengths), slots, max_seqlen=1200, z=layer.z,
                has_initial_state=init, y=y)
    assert (y[-9:] == 9).all() and cache.device_error() == m2.M2_ERR_BAD_SLOT
    check_scan(layer, cache, lengths[:-1], slots, init, y, before)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [m2.SelShape(256, 16, 1, 4, F32, BF16), m2.SelShape(1024, 16, 1, 4, BF16, BF16), m2.SelShape(2048, 16, 1, 4, F32, BF16),
                                   m2.SelShape(1024, 16, 1, 4, F32, F32), m2.SelShape(512, 32, 2, 4, F32, BF16), m2.SelShape(256, 64, 2, 4, F32, BF16),
                                   m2.SelShape(256, 8, 1, 4, F32, BF16)], ids=str)
def test_one_long_prompt(shape):
    """1100 tokens alone: two, four and eight states a lane in segments."""
    layer, cache = Layer(shape, 1100), cache_of(shape, 1)
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([1100]), ints(0), z=layer.z,
                    has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
    check_scan(layer, cache, [1100], ints(0), [1], y, before)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [512, 4096])
def test_scan_of_many_channels(D):
    """Enough channels for every way of spreading a channel's states over lanes."""
    shape = m2.SelShape(D, 16, 1, 4, F32, BF16)
    lengths = [40] * (4096 * 8 // D)
    layer = Layer(shape, sum(lengths))
    cache = cache_of(shape, len(lengths))
    slots = torch.arange(len(lengths), device="cuda", dtype=torch.int32)
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets(lengths), slots, max_seqlen=40, z=layer.z)
    some = [0, 3, len(lengths) - 1]
    cu = offsets(lengths)
    for i in some:
        ref, h, ysize, hsize = layer.reference(torch.zeros_like(before[i]), range(int(cu[i]), int(cu[i + 1])))
        within(y[cu[i]:cu[i + 1]], ref, ysize, 40, BF16, f"y {i}")
        within(cache.ssm[i], h, hsize, 40, F32, f"state {i}")


@pytest.mark.gpu
def test_scan_bad_slots_and_rows_behind():
    shape = m2.SelShape(64, 16, 1, 4, F32, BF16)
    lengths = [10, 20, 5]
    layer = Layer(shape, 40)  # five rows behind the last sequence
    cache = cache_of(shape, 3)
    before = cache.ssm.clone()
    y = torch.full((40, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets(lengths), ints(1, 3, 0), max_seqlen=20, z=layer.z, y=y)
    assert cache.device_error() == m2.M2_ERR_BAD_SLOT
    assert (y[10:30] == 9).all() and (y[35:] == 9).all()
    for i, (lo, hi, s) in enumerate(((0, 10, 1), (30, 35, 0))):
        ref, h, ysize, hsize = layer.reference(torch.zeros_like(before[s]), range(lo, hi))
        within(y[lo:hi], ref, ysize, hi - lo, BF16, f"y {i}")
        within(cache.ssm[s], h, hsize, hi - lo, F32, f"state {i}")
    assert torch.equal(cache.ssm[2], before[2])


@pytest.mark.gpu
def test_scan_of_strided_rows():
    """x and z as halves of one projection, B and C as slices of another."""
    shape = m2.SelShape(64, 16, 2, 4, F32, BF16)
    layer = Layer(shape, 50)
    cu, slots = offsets([20, 30]), ints(0, 1)
    cache, twin = cache_of(shape, 2), cache_of(shape, 2)
    want = m2.sel_scan(twin, layer.params, layer.x, layer.dt, layer.B, layer.C, cu, slots, z=layer.z)
    xz = torch.cat([layer.x, layer.z], 1)
    proj = torch.cat([torch.zeros(50, 8, dtype=torch.bfloat16, device="cuda"), layer.B.view(50, -1), layer.C.view(50, -1)], 1)
    out = torch.full((50, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    m2.sel_scan(cache, layer.params, xz[:, :64], layer.dt, proj[:, 8:40], proj[:, 40:72], cu, slots, z=xz[:, 64:], y=out[:, 16:80])
    assert torch.equal(out[:, 16:80], want) and (out[:, :16] == 3).all() and (out[:, 80:] == 3).all()
    assert torch.equal(cache.ssm, twin.ssm)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [60.0, 19.0, -12.0, -120.0])
def test_scan_at_the_ends_of_softplus(dt):
    """dt_raw far out: a state forgotten at once, one that barely moves, one that does not."""
    shape = m2.SelShape(32, 16, 1, 4, F32, F32)
    layer = Layer(shape, 12, z=False)
    layer.dt.fill_(dt)
    layer.params.dt_bias.zero_()
    cache = cache_of(shape, 1)
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([12]), ints(0),
                    has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
    check_scan(layer, cache, [12], ints(0), [1], y, before)
    one = cache_of(shape, 1)
    first = m2.sel_state_update(one, layer.params, layer.x[:1], layer.dt[:1], layer.B[:1], layer.C[:1], ints(0))
    ref, h, ysize, hsize = layer.reference(before[0], [0])
    within(first, ref, ysize, 1, F32, "y of the token")
    within(one.ssm[0], h, hsize, 1, F32, "state of the token")


@pytest.mark.gpu
def test_a_poisoned_channel_stays_alone():
    shape = m2.SelShape(64, 16, 1, 4, F32, BF16)
    layer = Layer(shape, 40)
    twin, cache = cache_of(shape, 2), cache_of(shape, 2)
    cu, slots = offsets([25, 15]), ints(0, 1)
    want = m2.sel_scan(twin, layer.params, layer.x, layer.dt, layer.B, layer.C, cu, slots, z=layer.z)
    layer.x[11, 5] = float("nan")
    layer.x[30, 9] = float("inf")
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, cu, slots, z=layer.z)
    bad = torch.zeros(40, 64, dtype=torch.bool, device="cuda")
    bad[11:25, 5] = bad[30:, 9] = True
    assert torch.equal(y[~bad], want[~bad]) and not torch.isfinite(y[11:25, 5]).any()
    assert torch.isnan(cache.ssm[0, 5]).all() and torch.equal(cache.ssm[0, :5], twin.ssm[0, :5])


# ---- tokens ----------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 5, 130])
@pytest.mark.parametrize("shape", SHAPES + [m2.SelShape(4096, 16, 1, 4, BF16, BF16)], ids=str)
def test_tokens(shape, batch):
    layer = Layer(shape, batch, z=batch != 5)
    cache = cache_of(shape, 140)
    slots = torch.randperm(140, device="cuda")[:batch].to(torch.int32)
    if batch > 1:
        slots[1] = -1
    before = cache.ssm.clone()
    y = m2.sel_state_update(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, slots, z=layer.z)
    check_scan(layer, cache, [1] * batch if batch < 8 else [1] * 8, slots[:8], [1] * 8, y, before) if batch < 8 else None
    if batch >= 8:
        for i in (0, 2, 77, batch - 1):
            ref, h, ysize, hsize = layer.reference(before[slots[i].long()], [i])
            within(y[i:i + 1], ref, ysize, 1, shape.act_dtype, f"y {i}")
            within(cache.ssm[slots[i].long()], h, hsize, 1, shape.state_dtype, f"state {i}")
        rest = torch.ones(140, dtype=torch.bool, device="cuda")
        rest[slots[slots >= 0].long()] = False
        assert torch.equal(cache.ssm[rest], before[rest]) and (y[1] == 0).all()
    slots[0] = 140
    m2.sel_state_update(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, slots, z=layer.z)
    assert cache.device_error() == m2.M2_ERR_BAD_SLOT


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_conv_of_prompts_and_tokens(act):
    """The conv over the D channels alone, and that its cache rolls: prompts, then a token."""
    shape = m2.SelShape(264, 16, 1, 4, F32, act)
    lengths = [2, 50, 0, 40]
    layer = Layer(shape, sum(lengths) + 4)
    cache = cache_of(shape, 5)
    before = cache.conv.clone()
    slots = ints(3, 0, 1, 4)
    T = sum(lengths)
    out = m2.sel_conv1d_update_varlen(cache, layer.taps, layer.x[:T], offsets(lengths), slots, 50)
    tokens = m2.sel_conv1d_update(cache, layer.taps, layer.x[T:], slots)
    cu = [0, 2, 52, 52, 92]
    w, b = layer.taps.weight.double(), layer.taps.bias.double()
    for i in range(4):
        raw = torch.cat([before[int(slots[i])], layer.x[cu[i]:cu[i + 1]], layer.x[T + i:T + i + 1]])
        pre = torch.einsum("tck,ck->tc", raw.double().unfold(0, 4, 1), w) + b
        size = torch.einsum("tck,ck->tc", raw.double().abs().unfold(0, 4, 1), w.abs()) + b.abs()
        want = pre * torch.sigmoid(pre)
        got = torch.cat([out[cu[i]:cu[i + 1]], tokens[i:i + 1]])
        # 16-bit outputs of long prompts take the tanh form of the SiLU, 2^-11 of the value's size
        bound = 1e-5 * size + (2.0 ** -8 * want.abs() + 2.0 ** -11 * pre.abs() if act == BF16 else 0)
        assert ((got.double() - want).abs() <= bound).all()
        assert torch.equal(cache.conv[int(slots[i])], raw[-3:])
    assert torch.equal(cache.conv[2], before[2])


@pytest.mark.gpu
def test_slots_past_32_bits():
    shape = m2.SelShape(8192, 16, 1, 4, F32, BF16)
    far = 2**31 // (8192 * 16) + 3  # its first element lies past 2^31
    big, small = m2.SelCache(shape, far + 1), cache_of(shape, 1)
    big.ssm[far], big.conv[far] = small.ssm[0], small.conv[0]
    layer = Layer(shape, 30)
    one = torch.ones(1, dtype=torch.uint8, device="cuda")
    for cache, slot in ((big, far), (small, 0)):
        at = ints(slot)
        x = m2.sel_conv1d_update_varlen(cache, layer.taps, layer.x, offsets([30]), at, 30)
        y = m2.sel_scan(cache, layer.params, x, layer.dt, layer.B, layer.C, offsets([30]), at, z=layer.z, has_initial_state=one)
        y2 = m2.sel_state_update(cache, layer.params, x[:1], layer.dt[:1], layer.B[:1], layer.C[:1], at)
        if cache is big:
            want = (y, y2)
    assert torch.equal(y, want[0]) and torch.equal(y2, want[1])
    assert torch.equal(big.ssm[far], small.ssm[0]) and torch.equal(big.conv[far], small.conv[0]) and not big.ssm[:far:4096].any()


@pytest.mark.gpu
def test_validate_mode_refuses_duplicates(monkeypatch):
    shape = m2.SelShape(64, 16, 1, 4, F32, BF16)
    layer, cache = Layer(shape, 4), cache_of(shape, 3)
    monkeypatch.setenv("M2_VALIDATE", "1")
    rest = (layer.x, layer.dt, layer.B, layer.C)
    with pytest.raises(m2.M2Error):
        m2.sel_scan(cache, layer.params, *rest, offsets([2, 2]), ints(1, 1))
    with pytest.raises(m2.M2Error):
        m2.sel_state_update(cache, layer.params, *(t[:2] for t in rest), ints(1, 1))
    with pytest.raises(m2.M2Error):
        m2.sel_conv1d_update(cache, layer.taps, layer.x[:2], ints(2, 2))
    m2.sel_scan(cache, layer.params, *rest, offsets([2, 2]), ints(1, -1))


@pytest.mark.gpu
def test_scans_on_two_streams_and_in_a_graph():
    """Segmented scans (clusters) beside each other, and captured: the same bits as in turn."""
    shape = m2.SelShape(128, 16, 1, 4, F32, BF16)
    layers = [Layer(shape, 900, seed=s) for s in (1, 2)]
    cu, slots = offsets([900]), ints(0)
    run = lambda i, c, **kw: m2.sel_scan(c, layers[i].params, layers[i].x, layers[i].dt, layers[i].B, layers[i].C, cu, slots,  # noqa: E731
                                         z=layers[i].z, has_initial_state=one, **kw)
    one = torch.ones(1, dtype=torch.uint8, device="cuda")
    first, second = [cache_of(shape, 1, s) for s in (1, 2)], [cache_of(shape, 1, s) for s in (1, 2)]
    want = [[run(i, first[i]) for _ in range(3)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(2):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(i, second[i]))
    torch.cuda.synchronize()
    y = torch.empty_like(want[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(0, second[0], y=y)
    graph.replay()
    assert torch.equal(y, want[0][2])
    run(1, second[1])
    for i in range(2):
        assert all(torch.equal(u, v) for u, v in zip(got[i], want[i])) and torch.equal(first[i].ssm, second[i].ssm)


@pytest.mark.gpu
@pytest.mark.parametrize("channels,act,out", [(8, BF16, torch.float32), (12, F32, torch.bfloat16)], ids=["bf16", "f32"])
def test_conv_of_few_channels(channels, act, out):
    """A vector or three of channels, a long prompt and a short one; outputs of another type in a wider buffer."""
    shape = m2.SelShape(channels, 16, 1, 4, F32, act)
    layer, cache = Layer(shape, 72), cache_of(shape, 2)
    before, buffer = cache.conv.clone(), torch.full((72, 16), 7.0, dtype=out, device="cuda")
    got = m2.sel_conv1d_update_varlen(cache, layer.taps, layer.x, offsets([70, 2]), ints(1, 0), 70, out=buffer[:, :channels])
    for slot, x, y in ((1, layer.x[:70], got[:70]), (0, layer.x[70:], got[70:])):
        raw = torch.cat([before[slot], x])
        pre = torch.einsum("tck,ck->tc", raw.double().unfold(0, 4, 1), layer.taps.weight.double()) + layer.taps.bias.double()
        want = pre * torch.sigmoid(pre)
        size = torch.einsum("tck,ck->tc", raw.double().abs().unfold(0, 4, 1), layer.taps.weight.double().abs()) + layer.taps.bias.double().abs()
        # 1e-5 of the sum's size for its fp32 terms and the SiLU, half a step of the output type
        assert ((y.double() - want).abs() <= 1e-5 * size + torch.finfo(out).eps / 2 * want.abs()).all()
        assert torch.equal(cache.conv[slot], raw[-3:])
    assert (buffer[:, channels:] == 7).all()


# ---- the path as it is used ------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_then_tokens_as_one_sequence(act):
    """A mixer as a model runs it: conv, the projections of its output to dt, B
    and C, the scan; prompts of different lengths, then three tokens a sequence,
    the last of them replayed from a captured graph. The states have to be those
    of the recurrence over the whole sequence on the same projections."""
    shape = m2.SelShape(128, 16, 1, 4, F32, act)
    lengths, more = [37, 64, 5], 3
    layer = Layer(shape, 1)
    g = torch.Generator(device="cuda").manual_seed(9)
    dtype = TYPES[act]
    draw = lambda *s, std=1.0: torch.empty(s, dtype=dtype, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    w_bc, w_dt = draw(128, 32, std=0.1), draw(128, 128, std=0.1)
    raw, z = draw(sum(lengths) + 3 * more, 128), draw(sum(lengths) + 3 * more, 128)
    cache = m2.SelCache(shape, 4)
    slots = ints(2, 0, 3)
    seen = []  # what the scan and the tokens read and wrote: (sequence, x, dt, B, C, z, y)

    def mix(x):
        bc = x @ w_bc
        return x @ w_dt, bc[:, :16], bc[:, 16:]

    T = sum(lengths)
    cu = offsets(lengths)
    x = m2.sel_conv1d_update_varlen(cache, layer.taps, raw[:T], cu, slots, 64)
    dt, B, C = mix(x)
    y = m2.sel_scan(cache, layer.params, x, dt, B, C, cu, slots, max_seqlen=64, z=z[:T])
    for i in range(3):
        r = slice(int(cu[i]), int(cu[i + 1]))
        seen.append([[t[r]] for t in (x, dt, B, C, z, y)])
    token, gate = torch.empty(3, 128, dtype=dtype, device="cuda"), torch.empty(3, 128, dtype=dtype, device="cuda")

    def step():
        xt = m2.sel_conv1d_update(cache, layer.taps, token, slots)
        d, b, c = mix(xt)
        return xt, d, b, c, gate, m2.sel_state_update(cache, layer.params, xt, d, b, c, slots, z=gate)

    graph = None
    for t in range(more):
        token.copy_(raw[T + 3 * t: T + 3 * t + 3])
        gate.copy_(z[T + 3 * t: T + 3 * t + 3])
        if t < more - 1:
            got = step()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step()
            graph.replay()
        for i in range(3):
            for to, v in zip(seen[i], got):
                to.append(v[i:i + 1].clone())
    for i, n in enumerate(lengths):
        xs, ds, Bs, Cs, zs, ys = (torch.cat(v) for v in seen[i])
        layer.x, layer.dt, layer.B, layer.C, layer.z = xs, ds, Bs[:, None], Cs[:, None], zs
        ref, h, ysize, hsize = layer.reference(torch.zeros(128, 16, device="cuda"), range(n + more))
        within(ys, ref, ysize, n + more, act, f"y of sequence {i}")
        within(cache.ssm[int(slots[i])], h, hsize, n + more, F32, f"state of sequence {i}")
        # the conv saw the sequence as one
        whole = torch.cat([torch.zeros(3, 128, dtype=dtype, device="cuda"), raw[int(cu[i]):int(cu[i + 1])],
                           *[raw[T + 3 * t + i][None] for t in range(more)]])
        assert torch.equal(cache.conv[int(slots[i])], whole[-3:])
    assert (cache.ssm[1] == 0).all() and cache.device_error() == 0


@pytest.mark.gpu
def test_a_prompt_in_two_parts_is_the_whole():
    shape = m2.SelShape(96, 16, 1, 4, F32, F32)
    layer = Layer(shape, 100)
    whole, parts = cache_of(shape, 1), cache_of(shape, 1)
    one = torch.ones(1, dtype=torch.uint8, device="cuda")
    want = m2.sel_scan(whole, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([100]), ints(0), z=layer.z, has_initial_state=one)
    got = []
    for lo, hi in ((0, 41), (41, 100)):
        got.append(m2.sel_scan(parts, layer.params, *(t[lo:hi] for t in (layer.x, layer.dt, layer.B, layer.C)), offsets([hi - lo]), ints(0),
                               z=layer.z[lo:hi], has_initial_state=one))
    size = layer.reference(cache_of(shape, 1).ssm[0], range(100))
    within(torch.cat(got), want.double(), size[2], 100, F32, "y")
    within(parts.ssm[0], whole.ssm[0].double(), size[3], 100, F32, "state")


@pytest.mark.gpu
@pytest.mark.parametrize("shape,T,n", [(m2.SelShape(64, 16, 1, 4, F32, BF16), 256, 16), (m2.SelShape(16, 16, 1, 4, F32, BF16), 512, 16),
                                       (m2.SelShape(64, 16, 1, 4, F32, F32), 250, 16), (m2.SelShape(16, 128, 2, 4, BF16, BF16), 128, 8),
                                       (m2.SelShape(16, 64, 1, 4, F32, F32), 1000, 8)], ids=str)
def test_segments_start_from_the_initial_state(shape, T, n):
    """Every segment of a sequence reads the slot's state at the start of the
    call, though the last one leaves the new state there: with a tile or two a
    segment, over and over on the same inputs, the same bits, and those of the
    recurrence. (States of 50 in size: a segment that began from the final state
    would be far off.)"""
    layer, cache = Layer(shape, n * T, seed=11), cache_of(shape, n, seed=12)
    cache.ssm.mul_(500)
    before = cache.ssm.clone()
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    one = torch.ones(n, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(40):
        cache.ssm.copy_(before)
        y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([T] * n), slots, max_seqlen=T, z=layer.z,
                        has_initial_state=one)
        if first is None:
            first = (y, cache.ssm.clone())
        assert torch.equal(y, first[0]) and torch.equal(cache.ssm, first[1])
    for i in (0, n - 1):
        s, rows = int(slots[i]), range(i * T, (i + 1) * T)
        ref, h, ysize, hsize = layer.reference(before[s], rows)
        within(y[i * T:(i + 1) * T], ref, ysize, T, shape.act_dtype, f"y of sequence {i}")
        within(cache.ssm[s], h, hsize, T, shape.state_dtype, f"state of sequence {i}")


def test_too_many_tokens_are_refused_on_the_host():
    """A kernel's token numbers have 32 bits and run past the last token by what its
    CTAs have in flight: a call takes 2^31 - 2^24 tokens at most."""
    L = m2.lib()
    s = m2.SelShape(8, 8, 1, 4, F32, BF16).c()
    cache = m2.m2_sel_cache()
    assert L.m2_sel_cache_wrap(ctypes.byref(s), 4, 0x100000, 0x200000, None, ctypes.byref(cache)) == m2.M2_OK
    p, taps, buf = m2.m2_sel_params(0x300000, 0x300100, 0x300200), m2.m2_conv_params(0x500000, None, 1), 0x400000

    def scan(total):  # (x is missing: no call gets past the checks)
        return L.m2_sel_scan(ctypes.byref(cache), ctypes.byref(p), 1, buf, total, 5, None, 8, buf, 8, buf, 8, buf, 8, None, 0, buf, 8, buf, None, None)

    def conv(total):
        return L.m2_sel_conv1d_update_varlen(ctypes.byref(cache), ctypes.byref(taps), 1, buf, total, 5, None, 8, buf, BF16, 8, buf, None)

    def conv_rows(batch, seqlen):
        return L.m2_sel_conv1d_update(ctypes.byref(cache), ctypes.byref(taps), batch, seqlen, None, 8, buf, BF16, 8, buf, None)

    most = 2**31 - 2**24
    for call in (scan, conv):
        for total in (most + 1, 2**31 - 100, 2**31 - 1, 2**31):
            assert call(total) == m2.M2_ERR_UNSUPPORTED, (call, total)
        assert call(most) == m2.M2_ERR_INVALID_ARG  # not refused for its size, but for what is missing
    assert conv_rows(1, most + 1) == m2.M2_ERR_UNSUPPORTED and conv_rows(2**15, 2**16 - 1) == m2.M2_ERR_UNSUPPORTED
    assert conv_rows(1, most) == m2.M2_ERR_INVALID_ARG


def bf16_values(low, high):
    """Every bf16 value between low and high that is no denormal."""
    v = torch.arange(-2**15, 2**15).to(torch.int16).view(torch.bfloat16).float()
    v = v[torch.isfinite(v) & (v >= low) & (v <= high) & ((v.abs() >= 2.0 ** -20) | (v == 0))]
    return v.unique().cuda()


def grid_rows(values, D):
    """The values as rows of D, the last one filled up."""
    return torch.cat([values, values[-1:].expand(-len(values) % D)]).view(-1, D)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_the_gate_from_far_below_to_far_above(act):
    """y = x silu(z) for every bf16 z of -80 .. 80 (C = 0, D = 1), rounded once, of a
    prompt and of tokens. The SiLU has an exponential, a sum, a reciprocal and a
    product or two; -z log2(e) is rounded by 2^-24 of up to 116, which is 80 * 2^-24 of
    the exponential, and its constant by 1.4e-8: 80 * 1.3 * 2^-24 + 4 * 2^-22 = 7.2e-6
    in all."""
    D = 64
    shape = m2.SelShape(D, 16, 1, 4, F32, act)
    z = grid_rows(bf16_values(-80.0, 80.0), D).to(TYPES[act])
    T = z.shape[0]
    layer = Layer(shape, T)
    layer.C.zero_()
    layer.params.D.fill_(1)
    layer.x.copy_(torch.where(torch.arange(T, device="cuda")[:, None] % 2 == 0, 1.0, -3.0))
    layer.z = z
    gate = z.double() * torch.sigmoid(z.double())
    want = layer.x.double() * gate
    bound = (7.2e-6 + torch.finfo(TYPES[act]).eps / 2) * want.abs()
    cache = cache_of(shape, T)
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([T]), ints(0), z=z)
    off = ((y.double() - want).abs() / bound.clamp_min(1e-300)).max()
    assert off <= 1, f"prompt: {off:.3g} times the bound"
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    tokens = m2.sel_state_update(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, slots, z=z)
    off = ((tokens.double() - want).abs() / bound.clamp_min(1e-300)).max()
    assert off <= 1, f"tokens: {off:.3g} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_infinite_gates_stay_alone(act):
    """silu(inf) = inf and a NaN stays one, each in its own value of y; states are untouched by z."""
    shape = m2.SelShape(32, 16, 1, 4, F32, act)
    layer = Layer(shape, 6)
    plain, cache = cache_of(shape, 6), cache_of(shape, 6)
    want = m2.sel_scan(plain, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([6]), ints(0), z=layer.z)
    layer.z[2, 3], layer.z[4, 8] = float("inf"), float("nan")
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([6]), ints(0), z=layer.z)
    tokens = m2.sel_state_update(cache_of(shape, 6), layer.params, layer.x, layer.dt, layer.B, layer.C, ints(0, 1, 2, 3, 4, 5), z=layer.z)
    rest = torch.isfinite(layer.z)
    for got in (y, tokens):
        assert torch.isinf(got[2, 3]) and torch.isnan(got[4, 8]) and torch.isfinite(got[rest]).all()
    assert torch.equal(y[rest], want[rest]) and torch.equal(plain.ssm, cache.ssm)


def one_token_states(act, v, A_log, x, h0):
    """The fp32 states after one token of each row of v (dt_raw, its bias zero; B = 1), by sel_scan and by sel_state_update."""
    n, D = v.shape
    shape = m2.SelShape(D, 16, 1, 4, F32, act)
    dtype = TYPES[act]
    params = m2.SelParams(A_log.contiguous(), torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda"))
    xs = torch.full((n, D), x, dtype=dtype, device="cuda")
    B = torch.ones(n, 1, 16, dtype=dtype, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    got = []
    for scan in (True, False):
        cache = m2.SelCache(shape, n)
        cache.ssm.fill_(h0)
        if scan:
            m2.sel_scan(cache, params, xs, v.to(dtype), B, B, offsets([1] * n), slots, max_seqlen=1,
                        has_initial_state=torch.ones(n, dtype=torch.uint8, device="cuda"))
        else:
            m2.sel_state_update(cache, params, xs, v.to(dtype), B, B, slots)
        got.append(cache.ssm.double())
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_softplus_within_its_bound(act):
    """A state that one token starts from zero with x = B = 1 is dt itself, in fp32:
    within 5e-7 + |v| 2^-23 of softplus(v) for every bf16 v of -86 .. 80."""
    v = grid_rows(bf16_values(-86.0, 80.0), 64)
    want = torch.nn.functional.softplus(v.double(), threshold=60).clamp_min(0)
    want = torch.where(v < -30, v.double().exp(), want)[..., None]
    bound = (5e-7 + v.double().abs() * 2.0 ** -23)[..., None] * want
    for name, got in zip(("scan", "token"), one_token_states(act, v, torch.zeros(64, 16, device="cuda"), 1.0, 0.0)):
        off = ((got - want).abs() / bound).max()
        assert off <= 1, f"{name}: {off:.3g} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
def test_decays_within_their_bound(act):
    """A state of one that a token of x = 0 leaves is the decay exp(dt A): within
    3e-7 + |dt A| (1e-6 + (|v| + |A_log|) 2^-23) of itself."""
    v = grid_rows(bf16_values(-12.0, 6.0), 64)
    A_log = torch.linspace(-6, 4, 64 * 16, device="cuda").view(64, 16)
    dtA = torch.nn.functional.softplus(v.double(), threshold=40)[..., None] * A_log.double().exp()
    want = torch.exp(-dtA)
    bound = (3e-7 + dtA * (1e-6 + (v.double().abs()[..., None] + A_log.double().abs()) * 2.0 ** -23)) * want + 2.0 ** -125
    for name, got in zip(("scan", "token"), one_token_states(act, v, A_log, 0.0, 1.0)):
        off = ((got - want).abs() / bound).max()
        assert off <= 1, f"{name}: {off:.3g} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [60.0, 19.0, -12.0, -120.0])
@pytest.mark.parametrize("T", [12, 700], ids=["one run", "segments"])
def test_scan_of_16_bit_inputs_at_the_ends_of_softplus(dt, T):
    """As test_scan_at_the_ends_of_softplus, on the special-function unit's exponentials."""
    shape = m2.SelShape(32, 16, 1, 4, F32, BF16)
    layer = Layer(shape, T, z=False)
    layer.dt.fill_(dt)
    layer.params.dt_bias.zero_()
    cache = cache_of(shape, 1)
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([T]), ints(0),
                    has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
    check_scan(layer, cache, [T], ints(0), [1], y, before)
    one = cache_of(shape, 1)
    first = m2.sel_state_update(one, layer.params, layer.x[:1], layer.dt[:1], layer.B[:1], layer.C[:1], ints(0))
    ref, h, ysize, hsize = layer.reference(before[0], [0])
    within(first, ref, ysize, 1, BF16, "y of the token")
    within(one.ssm[0], h, hsize, 1, F32, "state of the token")


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [13, 777], ids=["one run", "segments"])
def test_states_that_forget_everything(act, T):
    """A_log of 100 and of +inf: such a state keeps its last token's addend alone,
    also where tokens past the sequence's end (dt = 0) share its last tile."""
    shape = m2.SelShape(24, 16, 1, 4, F32, act)
    layer = Layer(shape, T)
    layer.params.A_log[3, 5], layer.params.A_log[7, :8], layer.params.A_log[20] = float("inf"), 100.0, float("inf")
    cache = cache_of(shape, 3)
    before = cache.ssm.clone()
    y = m2.sel_scan(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, offsets([T]), ints(1), z=layer.z,
                    has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
    check_scan(layer, cache, [T], ints(1), [1], y, before)
    assert torch.isfinite(cache.ssm).all() and torch.isfinite(y).all()
    token = m2.sel_state_update(cache, layer.params, layer.x[:1], layer.dt[:1], layer.B[:1], layer.C[:1], ints(2), z=layer.z[:1])
    ref, h, ysize, hsize = layer.reference(before[2], [0])
    within(token, ref, ysize, 1, act, "y of the token")
    within(cache.ssm[2], h, hsize, 1, F32, "state of the token")


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 2, 9, 40])
@pytest.mark.parametrize("state", [BF16, F32], ids=["bf16", "f32"])
def test_tokens_row_by_row(batch, state):
    """Every row of a batch with padding rows in it, and every slot beside them."""
    shape = m2.SelShape(1040, 16, 2, 4, state, BF16)
    layer, cache = Layer(shape, batch), cache_of(shape, 50)
    slots = torch.randperm(50, device="cuda")[:batch].to(torch.int32)
    slots[1::4] = -1
    before = cache.ssm.clone()
    y = m2.sel_state_update(cache, layer.params, layer.x, layer.dt, layer.B, layer.C, slots, z=layer.z)
    check_scan(layer, cache, [1] * batch, slots, [1] * batch, y, before)
    assert cache.device_error() == 0
