"""Cases of the 8-bit state cache and of the per-channel selective scan.

``run`` computes a case either with the library (``own``) or in plain torch
operations; ``exact`` computes it in 64 bits. Four operators:

* ``park``    q8_store of n sequences from a 16- or 32-bit cache into an 8-bit
              one, and q8_load back into other slots (the values that the
              codes stand for are what comes back);
* ``fan``     q8_load alone: a few 8-bit snapshots of shared prefixes read
              into the slots of many sequences;
* ``decode``  q8_state_update for ``steps`` tokens of a batch on the 8-bit
              cache, whose states are then read back into a 16-bit cache (a
              verify step or a parked sequence wants them there);
* ``scan``    sel_scan over packed prompts, with the causal conv before it
              where ``conv`` is true; ``token`` is sel_state_update, the same
              for one token a sequence.

Lengths of packed prompts are a text, "2048,2048". Shapes: H heads of P rows of
N states in G groups with a conv of K taps; ``scan`` and ``token`` have D
channels of N states in G groups.
"""

import math

import torch

own = False

F32, BF16 = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
K = 4  # conv taps
CHUNK = 32  # tokens that the plain scan expands at a time


# ---------------------------------------------------------------- cases

def listed():
    mixer = dict(H=128, P=64, N=128, G=8)  # the Nemotron-H mixer layer of the benchmark
    return [
        # one preempted sequence leaves its slot and comes back: latency
        dict(name="park_one", op="park", n=1, slots=8, state="bf16", **mixer),
        # a batch of sequences is parked under memory pressure
        dict(name="park_batch", op="park", n=128, slots=192, state="bf16", **mixer),
        # four prefix snapshots start 96 sequences of the fp32-state layer
        dict(name="fan_out", op="fan", snapshots=4, n=96, slots=128, state="f32", H=64, P=64, N=128, G=8),
        # one sequence decodes: latency
        dict(name="decode_one", op="decode", batch=1, slots=8, steps=1, z=True, **mixer),
        # the benchmark's decode batch
        dict(name="decode_64", op="decode", batch=64, slots=96, steps=1, z=True, **mixer),
        # the largest serving batch of the benchmark, four tokens
        dict(name="decode_384", op="decode", batch=384, slots=400, steps=4, z=True, **mixer),
        # short ragged prompts and an empty one in a small fp32 model
        dict(name="scan_ragged", op="scan", D=512, N=16, G=1, lengths="1,0,7,130,33,257,64,2", act="f32", state="f32", z=True,
             initial=True, conv=True),
        # the benchmark's prefill batch
        dict(name="scan_batch", op="scan", D=8192, N=16, G=1, lengths=",".join(["2048"] * 8), act="bf16", state="bf16", z=True,
             initial=False, conv=False),
        # one long prompt of a narrow layer: few channels, many tokens
        dict(name="scan_long", op="scan", D=2048, N=16, G=1, lengths="16384", act="bf16", state="f32", z=True, initial=True,
             conv=False),
        # wide states in groups, odd lengths, with the conv
        dict(name="scan_wide", op="scan", D=4096, N=64, G=8, lengths="1000,37,611,1", act="bf16", state="bf16", z=False,
             initial=True, conv=True),
        # one sequence's token with the conv tap before it: latency
        dict(name="token_one", op="token", batch=1, slots=8, D=8192, N=16, G=1, act="bf16", state="bf16", z=True, conv=True),
        # a serving batch's token on fp32 states
        dict(name="token_256", op="token", batch=256, slots=300, D=8192, N=16, G=1, act="bf16", state="f32", z=True, conv=False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, evenly spread over the logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["park", "fan", "decode", "scan", "scan", "token"])
    state = rng.choice(["bf16", "f32"])
    if op in ("park", "fan", "decode"):
        G = rng.choice([1, 2, 4, 8])
        mixer = dict(H=G * rng.choice([4, 8, 16]), P=rng.choice([32, 64]), N=rng.choice([64, 128]), G=G)
        if op == "park":
            n = _spread(rng, 1, 128)
            return dict(op=op, n=n, slots=n + rng.randint(1, 40), state=state, **mixer)
        if op == "fan":
            n = _spread(rng, 1, 96)
            return dict(op=op, snapshots=rng.randint(1, 8), n=n, slots=n + rng.randint(0, 30), state=state, **mixer)
        batch = _spread(rng, 1, 320)
        return dict(op=op, batch=batch, slots=batch + rng.randint(0, 40), steps=rng.randint(1, 4), z=rng.random() < 0.7, **mixer)
    act = rng.choice(["bf16", "bf16", "f32"])
    G = rng.choice([1, 1, 2, 4])
    D = 8 * G * _spread(rng, 8, 1024 // G)
    N = rng.choice([8, 16, 16, 16, 32, 64])
    conv = rng.random() < 0.5
    if conv and act == "bf16":
        state = "bf16"  # a state is no more exact than the 16-bit conv output that it takes in
    if op == "token":
        batch = max(1, min(_spread(rng, 1, 256), (1 << 25) // (D * N)))
        return dict(op=op, batch=batch, slots=batch + rng.randint(0, 60), D=D, N=N, G=G, act=act, state=state, z=rng.random() < 0.7,
                    conv=conv)
    total = max(1, min(_spread(rng, 1, 16384), (1 << 30) // (D * N)))
    parts = rng.randint(1, 8)
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    lengths = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))
    return dict(op=op, D=D, N=N, G=G, lengths=lengths, act=act, state=state, z=rng.random() < 0.7, initial=rng.random() < 0.7,
                conv=conv)


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("park", "fan", "decode"):
        H, P, N, G = (case[k] for k in "HPNG")
        rows, cd = H * P, H * P + 2 * G * N
        q8 = rows * (N + 4)  # codes and one fp32 scale a row
        if op == "decode":
            conv = (K - 1) * cd * 2
            step = 2 * q8 + 2 * conv + 2 * cd + 2 * H + (2 if case["z"] else 1) * 2 * rows
            back = rows * N * 2 + conv  # what is read back has just been written
            fixed = cd * (K + 1) * 2 + 12 * H
            b, s = case["batch"], case["steps"]
            return {"bytes": b * (s * step + back) + s * fixed, "flops": b * s * rows * N * 6.0}
        sb = 4 if case["state"] == "f32" else 2
        full, conv = rows * N * sb, (K - 1) * cd * 2
        if op == "park":
            return {"bytes": case["n"] * (2 * full + q8 + 3 * conv), "flops": case["n"] * rows * N * 3.0}
        return {"bytes": case["snapshots"] * (q8 + conv) + case["n"] * (full + conv), "flops": case["n"] * rows * N * 1.0}
    D, N, G = (case[k] for k in "DNG")
    ab, sb = (4 if case[k] == "f32" else 2 for k in ("act", "state"))
    lengths = [int(v) for v in case["lengths"].split(",")] if op == "scan" else [1] * case["batch"]
    T = sum(lengths)
    live = sum(v > 0 for v in lengths)
    rows = (3 + bool(case["z"]) + bool(case["conv"])) * D + 2 * G * N  # x, dt, y, z, and the conv's input beside its output
    reads = 2 if op == "token" or case["initial"] else 1
    size = T * rows * ab + live * reads * D * N * sb + D * N * 4 + 8 * D
    if case["conv"]:
        size += live * 2 * (K - 1) * D * ab + D * (K + 1) * ab
    return {"bytes": size, "flops": T * D * (N * 6.0 + 12)}


# ---------------------------------------------------------------- inputs

class _Draws:
    """Normal and uniform tensors from one seed, on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, shape, std=1.0, dtype=torch.float32):
        v = torch.empty(shape, dtype=dtype, device="cuda")
        return v.normal_(0.0, std, generator=self.g)

    def uniform(self, shape, low, high):
        return torch.empty(shape, device="cuda").uniform_(low, high, generator=self.g)

    def order(self, n, count):
        """`count` different slots of n, as int32."""
        return torch.randperm(n, generator=self.g, device="cuda")[:count].to(torch.int32)


def _inputs(case, seed):
    """The tensors of a case, with the distributions of the library's workloads:
    activations N(0, 1), states N(0, 0.1), A = -U[1, 16], dt_bias the inverse
    softplus of U[1e-3, 0.1], conv weights N(0, 0.5)."""
    r = _Draws(seed)
    op = case["op"]
    s = {}

    def params(heads, a_shape):
        s["A_log"] = torch.log(r.uniform(a_shape, 1.0, 16.0))
        s["dt_bias"] = torch.log(torch.expm1(r.uniform((heads,), 1e-3, 0.1)))
        s["D"] = r.normal((heads,))

    def taps(channels, dtype):
        s["conv_w"] = r.normal((channels, K), 0.5, dtype)
        s["conv_b"] = r.normal((channels,), 0.1, dtype)

    if op in ("park", "fan", "decode"):
        H, P, N, G = (case[k] for k in "HPNG")
        cd = H * P + 2 * G * N
        slots = case["slots"]
        if op == "park":
            n = case["n"]
            # rows of unlike sizes: a head's scale differs by up to a factor of 30
            s["ssm"] = r.normal((slots, H, P, N), 0.1, TYPES[case["state"]])
            s["ssm"].mul_(r.uniform((slots, H, 1, 1), 0.1, 3.0).to(TYPES[case["state"]]))
            s["conv"] = r.normal((slots, K - 1, cd), 1.0, torch.bfloat16)
            s["src"], s["dst"], s["back"] = r.order(slots, n), r.order(n, n), r.order(slots, n)
            s["q"] = torch.zeros((n, H, P, N), dtype=torch.int8, device="cuda")
            s["scale"] = torch.zeros((n, H, P), device="cuda")
            s["q_conv"] = torch.zeros((n, K - 1, cd), dtype=torch.bfloat16, device="cuda")
            return s
        have = case["snapshots"] if op == "fan" else slots
        s["q"] = r.uniform((have, H, P, N), -127.49, 127.49).round_().to(torch.int8)
        s["scale"] = r.uniform((have, H, P), 1e-4, 4e-3)
        s["q_conv"] = r.normal((have, K - 1, cd), 1.0, torch.bfloat16)
        if op == "fan":
            n, dtype = case["n"], TYPES[case["state"]]
            s["src"] = torch.randint(0, have, (n,), generator=r.g, device="cuda", dtype=torch.int32)
            s["dst"] = r.order(slots, n)
            s["ssm"] = torch.zeros((slots, H, P, N), dtype=dtype, device="cuda")
            s["conv"] = torch.zeros((slots, K - 1, cd), dtype=torch.bfloat16, device="cuda")
            return s
        b, dtype = case["batch"], torch.bfloat16
        params(H, (H,))
        taps(cd, dtype)
        s["slots"], s["back"] = r.order(slots, b), r.order(b, b)
        s["xBC"] = r.normal((case["steps"], b, cd), 1.0, dtype)
        s["dt"] = r.normal((case["steps"], b, H), 1.0, dtype)
        s["z"] = r.normal((case["steps"], b, H * P), 1.0, dtype) if case["z"] else None
        s["ssm"] = torch.zeros((b, H, P, N), dtype=dtype, device="cuda")
        s["conv"] = torch.zeros((b, K - 1, cd), dtype=dtype, device="cuda")
        return s

    D, N, G = (case[k] for k in "DNG")
    dtype = TYPES[case["act"]]
    params(D, (D, N))
    if op == "scan":
        lengths = [int(v) for v in case["lengths"].split(",")]
        ends = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        T, n = ends[-1], len(lengths)
        slots = n + 2
        s["flags"] = torch.tensor([i % 3 != 2 for i in range(n)], dtype=torch.uint8, device="cuda") if case["initial"] else None
    else:
        T, n, slots = case["batch"], case["batch"], case["slots"]
    s["slots"] = r.order(slots, n)
    s["ssm"] = r.normal((slots, D, N), 0.1, TYPES[case["state"]])
    s["x"], s["dt"] = r.normal((T, D), 1.0, dtype), r.normal((T, D), 1.0, dtype)
    s["z"] = r.normal((T, D), 1.0, dtype) if case["z"] else None
    s["B"], s["C"] = r.normal((T, G, N), 1.0, dtype), r.normal((T, G, N), 1.0, dtype)
    s["conv"] = r.normal((slots, K - 1, D), 1.0, dtype)
    if case["conv"]:
        taps(D, dtype)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:  # the handles that a program keeps beside its tensors
        import mamba_recurrent_state_b200 as m2

        op = case["op"]
        if op in ("park", "fan", "decode"):
            kind = BF16 if op == "decode" or case["state"] == "bf16" else F32
            shape = m2.Shape(case["H"], case["P"], case["N"], case["G"], K, kind, BF16)
            s["cache"] = m2.Cache(shape, s["ssm"].shape[0], ssm=s["ssm"], conv=s["conv"])
            s["q8"] = m2.Q8Cache(shape, s["q"].shape[0], ssm=s["q"], scale=s["scale"], conv=s["q_conv"])
            if op == "decode":
                s["params"] = m2.SSMParams(s["A_log"], s["dt_bias"], s["D"])
        else:
            kind = {"f32": F32, "bf16": BF16}
            shape = m2.SelShape(case["D"], case["N"], case["G"], K, kind[case["state"]], kind[case["act"]])
            s["cache"] = m2.SelCache(shape, s["ssm"].shape[0], ssm=s["ssm"], conv=s["conv"])
            s["params"] = m2.SelParams(s["A_log"], s["dt_bias"], s["D"])
        if "conv_w" in s:
            s["taps"] = m2.ConvParams(s["conv_w"], s["conv_b"], 1)
        if op == "scan":
            s["longest"] = max(int(v) for v in case["lengths"].split(","))
    return s


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    import mamba_recurrent_state_b200 as m2

    case = s["case"]
    op = case["op"]
    if op == "park":
        m2.q8_store(s["cache"], s["q8"], s["src"], s["dst"])
        m2.q8_load(s["q8"], s["cache"], s["dst"], s["back"])
        return {"ssm": s["ssm"], "conv": s["conv"]}
    if op == "fan":
        m2.q8_load(s["q8"], s["cache"], s["src"], s["dst"])
        return {"ssm": s["ssm"], "conv": s["conv"]}
    if op == "decode":
        ys = []
        for t in range(case["steps"]):
            ys.append(m2.q8_state_update(s["q8"], s["params"], s["taps"], s["xBC"][t], s["dt"][t], s["slots"],
                                         z=s["z"][t] if case["z"] else None))
        m2.q8_load(s["q8"], s["cache"], s["slots"], s["back"])
        return {"y": ys, "ssm": s["ssm"], "conv": s["conv"]}
    x = s["x"]
    if op == "scan":
        if case["conv"]:
            x = m2.sel_conv1d_update_varlen(s["cache"], s["taps"], x, s["cu"], s["slots"], s["longest"])
        y = m2.sel_scan(s["cache"], s["params"], x, s["dt"], s["B"], s["C"], s["cu"], s["slots"], max_seqlen=s["longest"], z=s["z"],
                        has_initial_state=s["flags"])
    else:
        if case["conv"]:
            x = m2.sel_conv1d_update(s["cache"], s["taps"], x, s["slots"])
        y = m2.sel_state_update(s["cache"], s["params"], x, s["dt"], s["B"], s["C"], s["slots"], z=s["z"])
    return {"y": y, "x": x if case["conv"] else None, "ssm": s["ssm"], "conv": s["conv"] if case["conv"] else None}


# ---------------------------------------------------------------- plain form

def _codes(v):
    """Rows of fp32 values as int8 codes and scales. The product with the
    inverse is formed in 64 bits, where it is exact: a code next to a border
    goes by the definition."""
    a = v.abs().amax(-1, keepdim=True)
    live = (a >= 2.0 ** -100) & torch.isfinite(a)
    safe = torch.where(live, a, torch.ones_like(a))
    inv = torch.full_like(safe, 127.0) / safe
    scale = torch.where(live, safe / torch.full_like(safe, 127.0), torch.zeros_like(a))
    scale = torch.where(torch.isfinite(a), scale, torch.full_like(a, math.nan))
    q = torch.round(v.double() * inv.double())
    return torch.where(live, q, torch.zeros_like(q)).to(torch.int8), scale.squeeze(-1)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _conv_rows(history, x, w, b):
    """Conv and SiLU over [n, t, channels] after the K-1 rows of `history`."""
    rows = torch.cat([history, x], 1).float()
    t = x.shape[1]
    out = b.float() + sum(rows[:, k : k + t] * w[:, k].float() for k in range(K))
    return _silu(out)


def _decode_plain(s, t):
    case = s["case"]
    H, P, N, G = (case[k] for k in "HPNG")
    slots, x = s["slots"].long(), s["xBC"][t]
    b = x.shape[0]
    history = s["q_conv"][slots]
    v = _conv_rows(history, x.unsqueeze(1), s["conv_w"], s["conv_b"])[:, 0]
    s["q_conv"][slots] = torch.cat([history[:, 1:], x.unsqueeze(1)], 1)
    xs = v[:, : H * P].view(b, H, P)
    B = v[:, H * P : H * P + G * N].view(b, G, N).repeat_interleave(H // G, 1)
    C = v[:, H * P + G * N :].view(b, G, N).repeat_interleave(H // G, 1)
    dt = _softplus(s["dt"][t].float() + s["dt_bias"])
    dA = torch.exp(dt * -torch.exp(s["A_log"]))
    S = s["q"][slots].float() * s["scale"][slots].unsqueeze(-1)
    S = S * dA[:, :, None, None] + (dt.unsqueeze(-1) * xs).unsqueeze(-1) * B.unsqueeze(2)
    y = (S * C.unsqueeze(2)).sum(-1) + s["D"][:, None] * xs
    y = y.reshape(b, H * P)
    if case["z"]:
        y = y * _silu(s["z"][t].float())
    s["q"][slots], s["scale"][slots] = _codes(S)
    return y.to(torch.bfloat16)


def _load_plain(s, src, dst):
    src, dst = src.long(), dst.long()
    s["ssm"][dst] = (s["q"][src].float() * s["scale"][src].unsqueeze(-1)).to(s["ssm"].dtype)
    s["conv"][dst] = s["q_conv"][src]


def _padded(s):
    """[sequences, longest] token numbers of packed prompts, and which are real."""
    cu = s["cu"].long()
    lengths = cu[1:] - cu[:-1]
    longest = max(int(v) for v in s["case"]["lengths"].split(","))
    at = torch.arange(longest, device="cuda")
    real = at < lengths[:, None]
    return torch.where(real, cu[:-1, None] + at, torch.zeros_like(real, dtype=torch.long)), real


def _scan_plain(s, x, at, real):
    """The scan over [n, T] tokens `at`: a chunk's factors are formed at once,
    the states one token after the other."""
    case = s["case"]
    D, N, G = (case[k] for k in "DNG")
    slots = s["slots"].long()
    n, T = at.shape
    A = -torch.exp(s["A_log"])
    h = s["ssm"][slots].float()
    if case["op"] == "scan":
        keep = s["flags"].bool() if s["flags"] is not None else torch.zeros(n, dtype=torch.bool, device="cuda")
        h = torch.where((keep | ~real.any(1))[:, None, None], h, torch.zeros_like(h))
    y = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    for t0 in range(0, T, CHUNK):
        i, m = at[:, t0 : t0 + CHUNK], real[:, t0 : t0 + CHUNK]
        xs = torch.where(m[..., None], x[i].float(), 0.0)
        dt = torch.where(m[..., None], _softplus(s["dt"][i].float() + s["dt_bias"]), 0.0)
        B = s["B"][i].float().repeat_interleave(D // G, 2)
        C = s["C"][i].float().repeat_interleave(D // G, 2)
        dA = torch.exp(dt.unsqueeze(-1) * A)
        states = (dt * xs).unsqueeze(-1) * B
        for t in range(i.shape[1]):
            h = torch.addcmul(states[:, t], dA[:, t], h, out=states[:, t])
        out = (states * C).sum(-1) + s["D"] * xs
        y[i[m]] = out[m]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["ssm"][slots] = h.to(s["ssm"].dtype)
    return y.to(x.dtype)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "park":
        src, dst = s["src"].long(), s["dst"].long()
        s["q"][dst], s["scale"][dst] = _codes(s["ssm"][src].float())
        s["q_conv"][dst] = s["conv"][src]
        _load_plain(s, s["dst"], s["back"])
        return {"ssm": s["ssm"], "conv": s["conv"]}
    if op == "fan":
        _load_plain(s, s["src"], s["dst"])
        return {"ssm": s["ssm"], "conv": s["conv"]}
    if op == "decode":
        ys = [_decode_plain(s, t) for t in range(case["steps"])]
        _load_plain(s, s["slots"], s["back"])
        return {"y": ys, "ssm": s["ssm"], "conv": s["conv"]}
    if op == "scan":
        at, real = _padded(s)
    else:
        at = torch.arange(case["batch"], device="cuda")[:, None]
        real = torch.ones_like(at, dtype=torch.bool)
    x = s["x"]
    if case["conv"]:
        slots = s["slots"].long()
        history = s["conv"][slots]
        raw = torch.where(real[..., None], x[at], torch.zeros((), dtype=x.dtype, device="cuda"))
        out = _conv_rows(history, raw, s["conv_w"], s["conv_b"]).to(x.dtype)
        rows = torch.cat([history, raw], 1)
        last = real.sum(1)[:, None] + torch.arange(K - 1, device="cuda")  # the K-1 rows that end at each sequence's last token
        s["conv"][slots] = rows.gather(1, last[..., None].expand(-1, -1, rows.shape[2]))
        x = torch.empty_like(x)
        x[at[real]] = out[real]
    y = _scan_plain(s, x, at, real)
    return {"y": y, "x": x if case["conv"] else None, "ssm": s["ssm"], "conv": s["conv"] if case["conv"] else None}


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------------- 64 bits

def _codes64(v):
    """Values of 64-bit rows as their 8-bit codes give them back, without
    rounding anything but the code itself; the scales are those of fp32."""
    a = v.abs().amax(-1, keepdim=True).float()
    scale, inv = (a.double() / 127).float().double(), (127 / a.double()).float().double()
    live = a >= 2.0 ** -100
    return torch.where(live, torch.round(v * torch.where(live, inv, 0.0)) * scale, 0.0)


def _sigmoid_gate(v):
    return v * torch.sigmoid(v)


def _decode64(s, case):
    H, P, N, G = (case[k] for k in "HPNG")
    f = {k: s[k].double() for k in ("A_log", "dt_bias", "D", "conv_w", "conv_b", "dt", "xBC")}
    hpg, steps = H // G, case["steps"]
    ssm, conv = s["ssm"].double(), s["conv"].double()
    ys = torch.empty((steps, case["batch"], H * P), dtype=torch.float64, device="cuda")
    for i, (slot, back) in enumerate(zip(s["slots"].tolist(), s["back"].tolist())):
        inputs = torch.cat([s["q_conv"][slot].double(), f["xBC"][:, i]])
        S = s["q"][slot].double() * s["scale"][slot].double()[..., None]
        for t in range(steps):
            v = _sigmoid_gate((inputs[t : t + K] * f["conv_w"].T).sum(0) + f["conv_b"])
            x, B, C = torch.split(v, [H * P, G * N, G * N])
            dt = torch.nn.functional.softplus(f["dt"][t, i] + f["dt_bias"], threshold=40.0)
            decay = torch.exp(-dt * f["A_log"].exp())
            S = S.view(G, hpg, P, N) * decay.view(G, hpg, 1, 1)
            S = S + torch.einsum("ghp,gn->ghpn", (dt[:, None] * x.view(H, P)).view(G, hpg, P), B.view(G, N))
            y = torch.einsum("ghpn,gn->ghp", S, C.view(G, N)).reshape(H, P) + f["D"][:, None] * x.view(H, P)
            ys[t, i] = y.reshape(-1) * (_sigmoid_gate(s["z"][t, i].double()) if case["z"] else 1.0)
            S = _codes64(S.reshape(H, P, N))
        ssm[back], conv[back] = S, inputs[steps:]
    return {"y": list(ys), "ssm": ssm, "conv": conv}


def _conv64(s, case, starts, ends):
    x = s["x"].double()
    cache = s["conv"].double()
    w, b = s["conv_w"].double(), s["conv_b"].double()
    out = torch.empty_like(x)
    for i, (lo, hi) in enumerate(zip(starts, ends)):
        if hi == lo:
            continue
        slot = int(s["slots"][i])
        rows = torch.cat([cache[slot], x[lo:hi]])
        out[lo:hi] = _sigmoid_gate(torch.einsum("tck,ck->tc", rows.unfold(0, K, 1), w) + b)
        cache[slot] = rows[-(K - 1) :]
    return out, cache


def _scan64(s, case, x, starts, ends):
    """All prompts as one scan of (factor, addend) pairs, doubling the distance
    from step to step, a block of channels at a time."""
    D, N, G = (case[k] for k in "DNG")
    T = x.shape[0]
    first = torch.zeros(T, dtype=torch.bool, device="cuda")
    y = torch.empty((T, D), dtype=torch.float64, device="cuda")
    ssm = s["ssm"].double()
    live = [i for i in range(len(starts)) if ends[i] > starts[i]]
    first[[starts[i] for i in live]] = True
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=40.0)
    keep = case["op"] == "token" or case["initial"]
    width = max(1, min(D // G, (1 << 27) // (T * N)))
    for g in range(G):
        B, C = s["B"][:, g].double()[:, None], s["C"][:, g].double()[:, None]
        for d0 in range(g * (D // G), (g + 1) * (D // G), width):
            d = slice(d0, min(d0 + width, (g + 1) * (D // G)))
            a = torch.exp(-dt[:, d, None] * s["A_log"][d].double().exp())
            v = (dt[:, d] * x[:, d])[..., None] * B
            for i in live:
                if keep and (s.get("flags") is None or bool(s["flags"][i])):
                    v[starts[i]] += a[starts[i]] * ssm[int(s["slots"][i]), d]
            a[first] = 0.0
            far = 1
            while far < T:
                v[far:] += a[far:] * v[:-far]
                a[far:] *= a[:-far].clone()
                far *= 2
            y[:, d] = (v * C).sum(-1) + s["D"][d].double() * x[:, d]
            for i in live:
                ssm[int(s["slots"][i]), d] = v[ends[i] - 1]
    if s["z"] is not None:
        y *= _sigmoid_gate(s["z"].double())
    return y, ssm


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("park", "fan"):
        ssm, conv = s["ssm"].double(), s["conv"].double()
        if op == "park":
            ssm[s["back"].long()] = _codes64(ssm[s["src"].long()])
            conv[s["back"].long()] = conv[s["src"].long()]
        else:
            ssm[s["dst"].long()] = (s["q"].double() * s["scale"].double()[..., None])[s["src"].long()]
            conv[s["dst"].long()] = s["q_conv"].double()[s["src"].long()]
        return {"ssm": ssm, "conv": conv}
    if op == "decode":
        return _decode64(s, case)
    if op == "scan":
        cu = s["cu"].tolist()
        starts, ends = cu[:-1], cu[1:]
    else:
        starts, ends = list(range(case["batch"])), list(range(1, case["batch"] + 1))
    x, cache = s["x"].double(), None
    seen = x
    if case["conv"]:
        x, cache = _conv64(s, case, starts, ends)
        seen = x.to(s["x"].dtype).double()  # the scan reads the conv's output as it is stored
    y, ssm = _scan64(s, case, seen, starts, ends)
    return {"y": y, "x": x if case["conv"] else None, "ssm": ssm, "conv": cache}
