"""The 8-bit state cache: codes and values against the definition, bit for
bit, and the decode step on it against a 64-bit computation that starts from
the same codes.

Bounds. With a = max |S'| of a row and scale = a / 127, a stored value is at
most scale / 2 from S': half a step of the code. What fp32 adds to it: S' is
formed from terms that carry a few roundings each (the conv's SiLU about 3 ulp,
softplus, exp, two products), under 1e-5 of the larger term in all, the
library's fp32 bound. The conv is a sum of K + 1 terms in fp32, off by at most
(K + 1) 2^-24 of their absolute sum c; with the SiLU's slope (1.1 at most) and
K = 8 that is 1.1 * 9 * 2^-24 c = 5.9e-7 c < 0.1 c * 1e-5. So a conv output v
counts as |v| + 0.1 c in the size of a term (where the K terms cancel, |v|
alone says nothing of its error). y has that bound too in fp32; in bf16 it is
rounded once, by at most 2^-8 of itself.
"""

import ctypes

import numpy as np
import pytest
import torch

import mamba_recurrent_state_b200 as m2

F32, BF16 = m2.M2_F32, m2.M2_BF16
FP32_SLACK = 1e-5
TYPES = {F32: torch.float32, BF16: torch.bfloat16}


def reference_codes(v):
    """Codes and scales of fp32 rows by the definition (the product in 64 bits is exact)."""
    a = v.abs().amax(-1)
    finite = torch.isfinite(a)
    live = finite & (a >= 2.0 ** -100)
    d = torch.where(live, a, torch.ones_like(a))
    scale = (d.double() / 127.0).float()
    inv = (127.0 / d.double()).float()
    q = torch.round(v.double() * inv.double()[..., None])
    q = torch.where(live[..., None], q, torch.zeros_like(q)).to(torch.int8)
    return q, torch.where(live, scale, torch.where(finite, torch.zeros_like(a), torch.full_like(a, float("nan")))), live


def special_rows(v):
    """Rows where quantising can go wrong, put over the first rows of v [.., N]."""
    flat = v.view(-1, v.shape[-1])
    big = torch.finfo(v.dtype).max
    rows = [torch.zeros(v.shape[-1]), torch.full((v.shape[-1],), 1e-38), torch.full((v.shape[-1],), 2.0 ** -100),
            torch.full((v.shape[-1],), -3.0), torch.full((v.shape[-1],), big / 4), torch.arange(v.shape[-1]) * 2.0 ** -90]
    one = torch.zeros(v.shape[-1])
    one[-1] = -7.5
    rows.append(one)
    ties = torch.arange(v.shape[-1]).float() / 2  # codes next to a border: multiples of half a step
    ties[0] = 127.0
    rows.append(ties)
    for i, r in enumerate(rows):
        flat[i] = r.to(v.dtype)
    return len(rows)


# ---- host: refusals ------------------------------------------------------------

def test_wrap_and_sizes_on_the_host():
    nemo = m2.Shape(128, 64, 128, 8, 4).c()
    out = m2.m2_q8_cache()
    L = m2.lib()
    n = [ctypes.c_int64() for _ in range(3)]
    assert L.m2_q8_cache_bytes(ctypes.byref(nemo), 2, *[ctypes.byref(v) for v in n]) == m2.M2_OK
    assert [v.value for v in n] == [2 * 2**20, 2 * 8192 * 4, 2 * 3 * 10240 * 2]
    assert L.m2_q8_cache_wrap(ctypes.byref(nemo), 4, 0x1000, 0x2000, 0x3000, None, ctypes.byref(out)) == m2.M2_OK
    for bad in ((0x1008, 0x2000, 0x3000), (0x1000, 0x2004, 0x3000), (0x1000, 0x2000, 0x3002), (None, 0x2000, 0x3000)):
        assert L.m2_q8_cache_wrap(ctypes.byref(nemo), 4, *bad, None, ctypes.byref(out)) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_cache_wrap(ctypes.byref(nemo), 0, 0x1000, 0x2000, 0x3000, None, ctypes.byref(out)) == m2.M2_ERR_INVALID_ARG
    for shape, want in ((m2.Shape(8, 64, 256, 1, 4, F32, F32), m2.M2_OK),  # an 8-bit state has one width
                        (m2.Shape(8, 64, 96, 1, 4), m2.M2_ERR_UNSUPPORTED), (m2.Shape(8, 12, 64, 1, 4), m2.M2_ERR_UNSUPPORTED),
                        (m2.Shape(256, 64, 128, 1, 4), m2.M2_ERR_UNSUPPORTED), (m2.Shape(8, 64, 128, 3, 4), m2.M2_ERR_INVALID_ARG),
                        (m2.Shape(8, 64, 128, 1, 9), m2.M2_ERR_UNSUPPORTED),
                        (m2.Shape(65536, 8, 64, 65536, 4), m2.M2_ERR_UNSUPPORTED)):
        s = shape.c()
        assert L.m2_q8_shape_check(ctypes.byref(s)) == want


def test_entry_points_refuse_bad_arguments():
    """Caches around made-up addresses: nothing of them is read on the host."""
    L = m2.lib()
    s = m2.Shape(128, 64, 128, 8, 4).c()
    q8, full = m2.m2_q8_cache(), m2.m2_cache()
    assert L.m2_q8_cache_wrap(ctypes.byref(s), 4, 0x100000, 0x200000, 0x300000, None, ctypes.byref(q8)) == m2.M2_OK
    assert L.m2_cache_wrap(ctypes.byref(s), 4, 0x400000, 0x500000, None, ctypes.byref(full)) == m2.M2_OK
    Q, Fc = ctypes.byref(q8), ctypes.byref(full)
    ssm, conv = m2.m2_ssm_params(0x600000, 0x600100, 0x600200), m2.m2_conv_params(0x700000, None, 1)
    buf, idx = 0x800000, 0x900000
    good = dict(ssm=ctypes.byref(ssm), conv=ctypes.byref(conv), batch=0, xBC=buf, xs=10240, dt=buf, ds=128, z=buf, zs=8192,
                y=buf, ys=8192, idx=idx, st=None)
    assert L.m2_q8_state_update(Q, *good.values()) == m2.M2_OK  # empty batch
    bad = [dict(batch=-1), dict(ssm=None, batch=1), dict(conv=None, batch=1), dict(batch=1, xBC=None), dict(batch=1, xBC=buf + 2),
           dict(batch=1, xs=10239), dict(batch=1, xs=10241), dict(batch=1, ds=127), dict(batch=1, zs=8191), dict(batch=1, z=buf + 4),
           dict(batch=1, y=None), dict(batch=1, ys=8193), dict(batch=1, idx=None)]
    for change in bad:
        assert L.m2_q8_state_update(Q, *{**good, **change}.values()) == m2.M2_ERR_INVALID_ARG, change
    assert L.m2_q8_state_update(Q, *{**good, "batch": 65536}.values()) == m2.M2_ERR_UNSUPPORTED
    assert L.m2_q8_state_update(None, *good.values()) == m2.M2_ERR_INVALID_ARG
    norm = m2.m2_norm_params(0x700100, -1.0)
    rest = list({**good, "batch": 1}.values())
    assert L.m2_q8_state_update_norm(Q, *rest[:2], ctypes.byref(norm), *rest[2:]) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_state_update_norm(Q, *rest[:2], None, *rest[2:]) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_store(Fc, Q, 0, None, None, None) == m2.M2_OK
    assert L.m2_q8_store(Fc, Q, 1, None, idx, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_store(Fc, Q, -1, idx, idx, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_load(Q, None, 1, idx, idx, None) == m2.M2_ERR_INVALID_ARG
    other = m2.Shape(128, 64, 128, 8, 4, BF16, F32).c()  # another activation type
    full2 = m2.m2_cache()
    assert L.m2_cache_wrap(ctypes.byref(other), 4, 0x400000, 0x500000, None, ctypes.byref(full2)) == m2.M2_OK
    assert L.m2_q8_store(ctypes.byref(full2), Q, 1, idx, idx, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_zero_slots(Q, -1, idx, None) == m2.M2_ERR_INVALID_ARG
    assert L.m2_q8_get_device_error(None, None, None) == m2.M2_ERR_INVALID_ARG


def test_binding_refuses_bad_tensors():
    shape = m2.Shape(8, 64, 128, 1, 4)
    q8 = m2.Q8Cache(shape, 4, device="cpu")
    act = torch.bfloat16
    params = m2.SSMParams(torch.zeros(8), torch.zeros(8), torch.zeros(8))
    taps = m2.ConvParams(torch.zeros(shape.conv_dim, 4, dtype=act), None)
    x, dt = torch.zeros(2, shape.conv_dim, dtype=act), torch.zeros(2, 8, dtype=act)
    slots = torch.zeros(2, dtype=torch.int32)
    for args in ((x.float(), dt, slots), (x[:, :-8], dt, slots), (x, dt[:1], slots), (x, dt, slots.long()), (x, dt, slots[:1])):
        with pytest.raises(ValueError):
            m2.q8_state_update(q8, params, taps, *args)
    with pytest.raises(ValueError, match="CUDA device"):
        m2.q8_state_update(q8, params, taps, x, dt, slots)
    with pytest.raises(ValueError):
        m2.Q8Cache(shape, 4, ssm=torch.zeros(4, 8, 64, 128))
    with pytest.raises(ValueError):
        m2.q8_store(q8, q8, slots, slots)


# ---- store and load --------------------------------------------------------------

def caches(shape, slots, q_slots, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = None
    if slots:
        full = m2.Cache(shape, slots)
        full.ssm.normal_(0.0, 0.1, generator=g)
        full.conv.normal_(0.0, 1.0, generator=g)
    q8 = m2.Q8Cache(shape, q_slots)
    q8.ssm.copy_(torch.randint(-127, 128, q8.ssm.shape, generator=g, device="cuda"))
    q8.scale.uniform_(1e-4, 1e-2, generator=g)
    q8.conv.normal_(0.0, 1.0, generator=g)
    return full, q8


COPY_SHAPES = [m2.Shape(8, 64, 128, 1, 4, BF16, BF16), m2.Shape(6, 24, 64, 3, 4, F32, F32), m2.Shape(5, 8, 256, 1, 2, BF16, F32),
               m2.Shape(64, 64, 128, 8, 4, F32, BF16), m2.Shape(4, 40, 64, 1, 8, BF16, BF16)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", COPY_SHAPES, ids=str)
def test_store_and_load_are_the_definition(shape):
    full, q8 = caches(shape, 6, 5)
    n_special = special_rows(full.ssm[4])
    src = torch.tensor([4, -1, 0, 5, 4], dtype=torch.int32, device="cuda")
    dst = torch.tensor([2, 0, 4, -1, 3], dtype=torch.int32, device="cuda")
    before = (q8.ssm.clone(), q8.scale.clone(), q8.conv.clone())
    m2.q8_store(full, q8, src, dst)
    for s, d in ((4, 2), (0, 4), (4, 3)):
        q, scale, _ = reference_codes(full.ssm[s].float())
        assert torch.equal(q8.ssm[d], q) and torch.equal(q8.scale[d], scale)
        assert torch.equal(q8.conv[d], full.conv[s])
    for d in (0, 1):  # untouched
        assert torch.equal(q8.ssm[d], before[0][d]) and torch.equal(q8.scale[d], before[1][d]) and torch.equal(q8.conv[d], before[2][d])
    values = q8.ssm[2].float() * q8.scale[2][..., None]
    live = reference_codes(full.ssm[4].float())[2]
    step = q8.scale[2][..., None].double()
    assert n_special and ((values.double() - full.ssm[4].double()).abs() <= step * (0.5 + 1e-4) + (~live[..., None]) * 2.0 ** -100).all()
    # read back: one snapshot into two slots
    keep = full.ssm[3].clone()
    back = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
    m2.q8_load(q8, full, torch.tensor([2, 2, 4], dtype=torch.int32, device="cuda"), back)
    for s, d in ((2, 1), (2, 0), (4, 2)):
        assert torch.equal(full.ssm[d], (q8.ssm[s].float() * q8.scale[s][..., None]).to(full.ssm.dtype))
        assert torch.equal(full.conv[d], q8.conv[s])
    assert torch.equal(full.ssm[3], keep)
    assert full.device_error() == 0 and q8.device_error() == 0


@pytest.mark.gpu
def test_rows_with_infinities_and_nans():
    shape = m2.Shape(8, 64, 128, 1, 4, F32, F32)
    full, q8 = caches(shape, 2, 2)
    full.ssm[0, 1, 3, 7], full.ssm[0, 2, 5, 0], full.ssm[0, 2, 6, 127] = float("inf"), float("nan"), float("-inf")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    m2.q8_store(full, q8, i, i)
    bad = torch.zeros(8, 64, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[2, 5] = bad[2, 6] = True
    assert torch.equal(torch.isnan(q8.scale[0]), bad)
    good = full.ssm[0][~bad].clone()
    m2.q8_load(q8, full, i, i)
    assert torch.isnan(full.ssm[0][bad]).all()
    assert ((full.ssm[0][~bad] - good).abs() <= q8.scale[0][~bad][..., None] * 0.5001).all()
    q8.zero_slots(i)
    m2.q8_load(q8, full, i, i)
    assert (full.ssm[0] == 0).all() and (full.conv[0] == 0).all()


@pytest.mark.gpu
def test_copies_report_bad_slots():
    shape = m2.Shape(8, 64, 128, 1, 4, BF16, BF16)
    full, q8 = caches(shape, 3, 2)
    before = q8.ssm.clone()
    at = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    m2.q8_store(full, q8, at(3, 1), at(0, 1))
    assert full.device_error() == m2.M2_ERR_BAD_SLOT and q8.device_error() == 0
    assert torch.equal(q8.ssm[0], before[0]) and torch.equal(q8.ssm[1], reference_codes(full.ssm[1].float())[0])
    m2.q8_load(q8, full, at(2), at(0))
    assert full.device_error() == 0 and q8.device_error() == m2.M2_ERR_BAD_SLOT


# ---- the decode step -------------------------------------------------------------

class Layer:
    """Parameters and rows of one mixer layer, and the step in 64 bits."""

    def __init__(self, shape, rows, seed=1, z=True, bias=True, activation=1, norm=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        act = TYPES[shape.act_dtype]
        draw = lambda *s, std=1.0, dt=act: torch.empty(s, dtype=dt, device="cuda").normal_(0, std, generator=g)  # noqa: E731
        uni = lambda n, lo, hi: torch.empty(n, device="cuda").uniform_(lo, hi, generator=g)  # noqa: E731
        self.shape, self.activation = shape, activation
        self.params = m2.SSMParams(uni(shape.H, 1, 16).log(), uni(shape.H, 1e-3, 0.1).expm1().log(), draw(shape.H, dt=torch.float32))
        self.taps = m2.ConvParams(draw(shape.conv_dim, shape.K, std=0.5), draw(shape.conv_dim, std=0.1) if bias else None, activation)
        hp = shape.H * shape.P
        self.norm = m2.NormParams(1 + draw(hp, std=0.1, dt=torch.float32).to(act), 1e-5) if norm else None
        self.xBC, self.dt = draw(rows, shape.conv_dim), draw(rows, shape.H)
        self.z = draw(rows, hp) if z else None

    def step(self, q, scale, conv, rows=slice(None)):
        """(y, S', size of S's terms) of `rows` from codes, scales and conv rows of their slots."""
        sh = self.shape
        H, P, N, G = sh.H, sh.P, sh.N, sh.G
        x64 = self.xBC[rows].double()
        b = x64.shape[0]
        win = torch.cat([conv.double(), x64[:, None]], 1)
        v = (win * self.taps.weight.double().T).sum(1)
        c = (win * self.taps.weight.double().T).abs().sum(1)
        if self.taps.bias is not None:
            v, c = v + self.taps.bias.double(), c + self.taps.bias.double().abs()
        if self.activation:
            v = v * torch.sigmoid(v)

        def parts(u):
            x, B, C = u.split([H * P, G * N, G * N], 1)
            return x.view(b, H, P), *(t.view(b, G, N).repeat_interleave(H // G, 1) for t in (B, C))

        x, B, C = parts(v)
        xs, Bs, Cs = parts(v.abs() + 0.1 * c)
        dt = torch.nn.functional.softplus(self.dt[rows].double() + self.params.dt_bias.double(), threshold=40)
        dA = torch.exp(dt * -self.params.A_log.double().exp())
        S = q.double() * scale.double()[..., None]
        decayed, fresh = S * dA[..., None, None], (dt[..., None] * x)[..., None] * B[:, :, None]
        new, size = decayed + fresh, decayed.abs() + (dt[..., None] * xs)[..., None] * Bs[:, :, None]
        y = (new * C[:, :, None]).sum(-1) + self.params.D.double()[:, None] * x
        ysize = (size * Cs[:, :, None]).sum(-1) + self.params.D.double().abs()[:, None] * xs
        y, ysize = y.reshape(b, -1), ysize.reshape(b, -1)
        if self.z is not None:
            gate = self.z[rows].double()
            gate = gate * torch.sigmoid(gate)
            y, ysize = y * gate, ysize * gate.abs()
        if self.norm is not None:
            grp = y.view(b, G, -1)
            r = torch.rsqrt(grp.square().mean(-1, keepdim=True) + self.norm.eps)
            w = self.norm.weight.double()
            y, ysize = (grp * r).view(b, -1) * w, (ysize.view(b, G, -1) * r).view(b, -1) * w.abs()
        return y, new, size, ysize

    def run(self, cache, slots, **kw):
        return m2.q8_state_update(cache, self.params, self.taps, self.xBC, self.dt, slots, z=self.z, norm=self.norm, **kw)


def check_step(layer, cache, slots, y, before, live=None):
    """y, codes, scales and conv rows after a step, against 64 bits from `before`."""
    live = range(len(slots)) if live is None else live
    at = slots[list(live)].long()
    q, scale, conv = (t[at] for t in before)
    ref_y, S, size, ysize = layer.step(q, scale, conv, list(live))
    got = cache.ssm[at].double() * cache.scale[at].double()[..., None]
    big = size.amax(-1, keepdim=True)
    off = (got - S).abs() - (cache.scale[at].double()[..., None] / 2 + FP32_SLACK * big)
    assert (off <= 0).all(), f"state off by {off.max():.3g} more than half a step"
    a = S.abs().amax(-1)
    assert ((cache.scale[at].double() * 127 - a).abs() <= FP32_SLACK * big[..., 0]).all()
    bound = FP32_SLACK * ysize
    if layer.shape.act_dtype == BF16:
        bound = bound + 2.0 ** -8 * ref_y.abs()
    worst = ((y[list(live)].double() - ref_y).abs() - bound).max()
    assert worst <= 0, f"y off by {worst:.3g} more than its bound"
    assert torch.equal(cache.conv[at], torch.cat([conv[:, 1:], layer.xBC[list(live)][:, None]], 1))


def snapshot(cache):
    return cache.ssm.clone(), cache.scale.clone(), cache.conv.clone()


UPDATE_SHAPES = [
    m2.Shape(128, 64, 128, 8, 4, BF16, BF16),  # the benchmark's layer: four CTAs a group
    m2.Shape(8, 64, 128, 1, 4, F32, F32),
    m2.Shape(6, 24, 64, 3, 4, BF16, BF16),     # a group shorter than one pass
    m2.Shape(9, 40, 64, 1, 3, BF16, F32),      # 360 rows: the last tile is short
    m2.Shape(4, 8, 256, 2, 2, F32, BF16),      # the smallest heads, the widest rows
    m2.Shape(128, 64, 128, 1, 4, BF16, BF16),  # one group of 8192 rows: 16 CTAs of 512
    m2.Shape(16, 256, 256, 1, 8, BF16, F32),   # one group of 4096 rows of 256
    m2.Shape(80, 8, 64, 1, 5, BF16, BF16),     # tiles that touch many heads
]


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("shape", UPDATE_SHAPES, ids=str)
def test_decode_steps(shape, norm):
    _, cache = caches(shape, 0, 7)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    for step in range(3):
        layer = Layer(shape, 3, seed=10 + step, z=step != 1, bias=step != 2, activation=int(step != 2), norm=norm)
        before = snapshot(cache)
        y = layer.run(cache, slots)
        check_step(layer, cache, slots, y, before)
        for s in (1, 2, 4, 6):
            assert torch.equal(cache.ssm[s], before[0][s]) and torch.equal(cache.scale[s], before[1][s]) and torch.equal(cache.conv[s], before[2][s])
    assert cache.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 2, 33, 150])
def test_decode_batches(batch):
    shape = m2.Shape(16, 32, 128, 2, 4, BF16, BF16)
    _, cache = caches(shape, 0, 160)
    slots = torch.randperm(160, device="cuda")[:batch].to(torch.int32)
    layer = Layer(shape, batch)
    before = snapshot(cache)
    check_step(layer, cache, slots, layer.run(cache, slots), before)


@pytest.mark.gpu
def test_decode_padding_and_bad_slots():
    shape = m2.Shape(16, 64, 128, 2, 4, BF16, BF16)
    _, cache = caches(shape, 0, 4)
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    layer = Layer(shape, 4)
    y = torch.full((4, 16 * 64), 9.0, dtype=torch.bfloat16, device="cuda")
    before = snapshot(cache)
    layer.run(cache, slots, y=y)
    check_step(layer, cache, slots, y, before, live=[0, 3])
    assert (y[1] == 0).all() and (y[2] == 9).all()
    assert torch.equal(cache.ssm[1], before[0][1]) and torch.equal(cache.ssm[3], before[0][3])
    assert cache.device_error() == m2.M2_ERR_BAD_SLOT and cache.device_error() == 0


@pytest.mark.gpu
def test_decode_of_strided_rows():
    shape = m2.Shape(8, 64, 128, 1, 4, BF16, BF16)
    _, cache = caches(shape, 0, 5)
    _, twin = caches(shape, 0, 5)
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    layer = Layer(shape, 2)
    want = layer.run(twin, slots)
    # z, xBC and dt as the columns of one projection, y inside a wider buffer
    hp, cd = 512, shape.conv_dim
    wide = torch.cat([layer.z, layer.xBC, layer.dt, torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")], 1)
    out = torch.full((2, hp + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    m2.q8_state_update(cache, layer.params, layer.taps, wide[:, hp:hp + cd], wide[:, hp + cd:hp + cd + 8], slots, z=wide[:, :hp],
                       y=out[:, 32:32 + hp])
    assert torch.equal(out[:, 32:32 + hp], want) and (out[:, :32] == 5).all() and (out[:, 32 + hp:] == 5).all()
    assert torch.equal(cache.ssm, twin.ssm) and torch.equal(cache.scale, twin.scale)


@pytest.mark.gpu
def test_decode_of_zero_and_poisoned_rows():
    """A zero state with a zero input stays zero; a NaN stays in its row and its y."""
    shape = m2.Shape(8, 64, 128, 1, 4, F32, F32)
    cache = m2.Q8Cache(shape, 2)
    layer = Layer(shape, 1, z=False, bias=False)
    layer.xBC.zero_()
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = layer.run(cache, slots)
    assert (y == 0).all() and (cache.ssm[0] == 0).all() and (cache.scale[0] == 0).all()
    layer = Layer(shape, 1, seed=4, z=False)
    cache.scale[0, 2, 5] = float("nan")
    y = layer.run(cache, slots)
    bad = torch.zeros(8, 64, dtype=torch.bool, device="cuda")
    bad[2, 5] = True
    assert torch.equal(torch.isnan(cache.scale[0]), bad) and torch.equal(torch.isnan(y[0].view(8, 64)), bad)


@pytest.mark.gpu
def test_decode_in_a_graph_and_on_another_stream():
    shape = m2.Shape(16, 64, 128, 2, 4, BF16, BF16)
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    layer = Layer(shape, 2)
    _, eager = caches(shape, 0, 3)
    want = [layer.run(eager, slots) for _ in range(4)]
    _, cache = caches(shape, 0, 3)
    full = m2.Cache(shape, 3)
    y = torch.empty_like(want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run(cache, slots, y=y)  # the first step
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # capturing runs nothing
        layer.run(cache, slots, y=y)
        m2.q8_load(cache, full, slots, slots)
    for i in range(1, 4):
        graph.replay()
        assert torch.equal(y, want[i])
    assert torch.equal(cache.ssm, eager.ssm) and torch.equal(cache.scale, eager.scale)
    assert torch.equal(full.ssm[0], (eager.ssm[0].float() * eager.scale[0][..., None]).bfloat16())


@pytest.mark.gpu
def test_slots_past_32_bits():
    """The last slot of a cache whose codes pass 2^31 bytes: the same bits as the first slot of a small one."""
    shape = m2.Shape(128, 64, 128, 8, 4, BF16, BF16)
    _, small = caches(shape, 0, 1)
    big = m2.Q8Cache(shape, 2100)
    last, zero = torch.tensor([2099], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for a, b in ((big.ssm, small.ssm), (big.scale, small.scale), (big.conv, small.conv)):
        a[2099] = b[0]
    layer = Layer(shape, 1)
    assert torch.equal(layer.run(big, last), layer.run(small, zero))
    full = m2.Cache(shape, 2)
    m2.q8_load(big, full, last, zero)
    m2.q8_store(full, big, zero, torch.tensor([2098], dtype=torch.int32, device="cuda"))
    want = m2.Cache(shape, 1)
    m2.q8_load(small, want, zero, zero)
    assert torch.equal(full.ssm[0], want.ssm[0]) and torch.equal(big.ssm[2098], reference_codes(want.ssm[0].float())[0])
    assert torch.equal(big.conv[2098], small.conv[0]) and not big.ssm[:2098].any()


@pytest.mark.gpu
def test_validate_mode_refuses_duplicates(monkeypatch):
    shape = m2.Shape(8, 64, 128, 1, 4, BF16, BF16)
    full, cache = caches(shape, 3, 3)
    layer = Layer(shape, 2)
    at = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    monkeypatch.setenv("M2_VALIDATE", "1")
    with pytest.raises(m2.M2Error):
        layer.run(cache, at(1, 1))
    with pytest.raises(m2.M2Error):
        m2.q8_store(full, cache, at(0, 1), at(2, 2))
    m2.q8_load(cache, full, at(2, 2), at(0, 1))  # a snapshot may be read twice
    layer.run(cache, at(1, -1))


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two batches on two caches on two streams, and again in turn: the same bits."""
    shape = m2.Shape(16, 64, 128, 2, 4, BF16, BF16)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    layers = [Layer(shape, 40, seed=s) for s in (1, 2)]
    pairs = [[caches(shape, 0, 40, seed=s)[1] for s in (1, 2)] for _ in range(2)]
    want = [[layers[i].run(pairs[0][i], slots) for _ in range(3)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(layers[i].run(pairs[1][i], slots))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(u, v) for u, v in zip(got[i], want[i]))
        assert torch.equal(pairs[0][i].ssm, pairs[1][i].ssm) and torch.equal(pairs[0][i].scale, pairs[1][i].scale)


# ---- the path as it is used ------------------------------------------------------

@pytest.mark.gpu
def test_prefill_park_decode_resume_verify():
    """Two prompts through the 16-bit cache, parked in 8 bits, decoded there for
    four tokens, read back, and two draft tokens verified on the 16-bit cache;
    against the same tokens on the 16-bit cache throughout.

    The two runs' states differ by the codes: half a step of each of five
    roundings, decayed in between, at most 5 * a / 254 of a row's maximum, and
    by the 16-bit run's own five roundings of 2^-9 (2^-8 at most) each. y is a
    sum of 128 such values times C: relative to its terms the same bound."""
    shape = m2.Shape(16, 64, 128, 2, 4, BF16, BF16)
    g = torch.Generator(device="cuda").manual_seed(3)
    T = 150
    layer = Layer(shape, 2 * T, seed=5)
    full, twin, q8 = m2.Cache(shape, 8), m2.Cache(shape, 8), m2.Q8Cache(shape, 4)
    home = torch.tensor([6, 1], dtype=torch.int32, device="cuda")
    away = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    for c in (full, twin):
        x = m2.conv1d_update(c, layer.taps, layer.xBC.view(2, T, -1), home, out_dtype=torch.float16)
        m2.chunk_scan(c, layer.params, x, layer.dt.view(2, T, -1), home, z=layer.z.view(2, T, -1))
    assert torch.equal(full.ssm, twin.ssm)
    m2.q8_store(full, q8, home, away)
    full.zero_slots(home)
    big = twin.ssm[home.long()].float().abs().amax(-1)
    for t in range(4):
        step = Layer(shape, 2, seed=20 + t)
        step.params, step.taps = layer.params, layer.taps
        ya = step.run(q8, away)
        yb = m2.state_update(twin, layer.params, step.xBC, step.dt, home, z=step.z, conv=layer.taps)
        big = torch.maximum(big, twin.ssm[home.long()].float().abs().amax(-1))
    m2.q8_load(q8, full, away, home)
    limit = 5 * (1 / 254 + 2.0 ** -8)
    assert ((full.ssm[home.long()].float() - twin.ssm[home.long()].float()).abs().amax(-1) <= limit * big).all()
    assert torch.equal(full.conv[home.long()], twin.conv[home.long()])
    drafts = Layer(shape, 4, seed=40)
    marks = torch.tensor([[0, 2], [3, 4]], dtype=torch.int32, device="cuda")
    ys = [m2.state_update_multi(c, layer.params, layer.taps, drafts.xBC.view(2, 2, -1), drafts.dt.view(2, 2, -1), home, marks,
                                z=drafts.z.view(2, 2, -1)) for c in (full, twin)]
    rel = lambda u, v: float((u.float() - v.float()).norm() / v.float().norm())  # noqa: E731
    assert rel(ya, yb) <= limit and rel(ys[0], ys[1]) <= limit
    assert q8.device_error() == 0 and full.device_error() == 0


def test_a_cache_is_described_on_the_device_of_its_tensors(monkeypatch):
    """Whatever device is current when the handle is made."""
    seen = []
    on = m2._on
    monkeypatch.setattr(m2, "_on", lambda device: (seen.append(device), on(device))[1])
    shape = m2.Shape(8, 64, 128, 1, 4)
    cache = m2.Cache(shape, 2, device="cpu")
    assert seen == [cache.ssm.device]


@pytest.mark.gpu
def test_copies_refuse_a_cache_of_another_device():
    """Either of the two caches described on a device that is not the current one:
    refused on the host, by the library itself."""
    shape = m2.Shape(8, 64, 128, 1, 4, BF16, BF16)
    full, q8 = caches(shape, 2, 2)
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    L, here = m2.lib(), full.c.device
    for handle in (full.c, q8.c):
        handle.device = here + 1
        rest = (1, i.data_ptr(), i.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert L.m2_q8_store(ctypes.byref(full.c), ctypes.byref(q8.c), *rest) == m2.M2_ERR_INVALID_ARG
        assert L.m2_q8_load(ctypes.byref(q8.c), ctypes.byref(full.c), *rest) == m2.M2_ERR_INVALID_ARG
        handle.device = here
    m2.q8_store(full, q8, i, i)
    assert torch.equal(q8.ssm[0], reference_codes(full.ssm[0].float())[0])


@pytest.mark.gpu
def test_the_largest_finite_values_read_back_finite():
    """127 times the rounded quotient of the largest float and 127 would be an infinity."""
    shape = m2.Shape(8, 64, 128, 1, 4, F32, F32)
    full, q8 = caches(shape, 2, 2)
    top = torch.finfo(torch.float32).max
    full.ssm[0, 0, 0, :4] = torch.tensor([top, -top, top / 2, 0.0])
    full.ssm[0, 0, 1, 5] = -top
    full.ssm[0, 0, 2, 0] = top * (1 - 2.0 ** -23)
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = full.ssm[0].clone()
    m2.q8_store(full, q8, i, i)
    m2.q8_load(q8, full, i, i)
    assert torch.isfinite(full.ssm[0]).all()
    # half a step, and the roundings to fp32 of scale, inverse and product
    step = q8.scale[0].double()[..., None]
    assert ((full.ssm[0].double() - want.double()).abs() <= step * (0.5 + 127 * 4 * 2.0 ** -24)).all()
    # and through a decode step that keeps the state: dt of zero, no input
    layer = Layer(shape, 1, z=False, bias=False)
    layer.xBC.zero_()
    layer.dt.fill_(-200)
    q8.conv.zero_()
    layer.run(q8, i)
    m2.q8_load(q8, full, i, i)
    assert torch.isfinite(full.ssm[0]).all()
    step = q8.scale[0].double()[..., None]
    assert ((full.ssm[0].double() - want.double()).abs() <= step * (0.5 + 127 * 6 * 2.0 ** -22)).all()
