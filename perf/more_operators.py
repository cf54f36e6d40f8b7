"""Cases, inputs and plain forms of the 8-bit and the expert-grouped products.

Five operators around N:M pruned weights in the PyTorch-linear layout:

  i8_quantize       rows -> 8-bit integers with one binary32 scale a row (a
                    token's activations, or an output channel's weights) and
                    back
  i8_linear         Y = act(X W^T + b): N:M packed 8-bit weights with a scale
                    for each channel, activations quantised by the call with a
                    scale for each token
  expert_linear     Y[s] = X[s] W_e^T for the rows s of each expert e, rows
                    sorted by expert, ragged counts, packed 16-bit weights
  expert_train      the same and its backward pass: dX, and dW where kept
  i8_expert_linear  the grouped product with 8-bit weights and activations

X is [T, K], weights [R, K] (experts: [E, R, K]), outputs [T, R]; expert e has
the rows offsets[e] .. offsets[e + 1] - 1, rows behind the last expert's belong
to none and come out as zeros.  A row's scale is amax / 127 rounded to
binary32, at least 2^-126; its elements are x / scale rounded half to even.
`run` computes the operators in their plain form with elementary torch
operations, or, where `own` is set, by the package's calls.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, T, R, K, dtype, E=0, N=2, M=4, act="none", pad=0, bias=False, rest=0):
    c = {"op": op, "T": T, "R": R, "K": K, "dtype": dtype, "E": E, "N": N, "M": M, "act": act, "pad": pad,
         "bias": bias, "rest": rest}
    if name is not None:
        c = {"name": name, **c}
    return c


def listed():
    return [
        # activations of one image, a width that is no whole vector
        _case("i8_quantize_197", "i8_quantize", 197, 0, 770, "bf16"),
        # a long prompt's activations in front of a down projection
        _case("i8_quantize_4096", "i8_quantize", 4096, 0, 11008, "fp16"),
        # one token of decoding through a pruned 7B-sized up projection
        _case("i8_linear_decode_1", "i8_linear", 1, 11008, 4096, "bf16"),
        # sixteen requests decoding together through the down projection, 4:8
        _case("i8_linear_decode_16_4of8", "i8_linear", 16, 4096, 11008, "fp16", N=4, M=8),
        # a short prompt through a small layer whose sizes fit no tile, its
        # activations a slice of a wider buffer, bias and GELU
        _case("i8_linear_ragged", "i8_linear", 77, 1500, 1000, "fp16", N=3, act="gelu", pad=5, bias=True),
        # a prompt of 2048 tokens: bound by the matrix cores
        _case("i8_linear_prompt_2048", "i8_linear", 2048, 11008, 4096, "bf16"),
        # eight requests decoding, two experts each of 32: many experts idle
        _case("expert_decode_16", "expert_linear", 16, 1536, 2048, "bf16", E=32),
        # a prompt of 2048 tokens, two experts each, the looser 4:8 pattern
        _case("expert_prompt_4of8", "expert_linear", 4096, 1536, 2048, "fp16", E=32, N=4, M=8),
        # one small training step, odd sizes, rows that no expert takes
        _case("expert_train_300", "expert_train", 300, 331, 500, "fp16", E=5, N=2, M=4, pad=3, rest=11),
        # one training step of eight experts on 4096 rows
        _case("expert_train_4096", "expert_train", 4096, 2048, 4096, "bf16", E=8),
        # the decoding requests through 8-bit experts
        _case("i8_expert_decode_16", "i8_expert_linear", 16, 1536, 2048, "bf16", E=32),
        # a prompt through 8-bit experts, a ragged number of rows
        _case("i8_expert_prompt_3900", "i8_expert_linear", 3900, 1536, 2048, "bf16", E=32, rest=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: rows, both widths and experts over their whole ranges."""
    op = rng.choice(["i8_quantize", "i8_linear", "i8_linear", "expert_linear", "expert_train", "i8_expert_linear"])
    N, M = rng.choice([(2, 4), (2, 4), (4, 8), (1, 4), (2, 8), (4, 4), (3, 4), (5, 8)])
    dtype, pad = rng.choice(["fp16", "bf16"]), rng.choice([0, 0, 8, 5])
    if op == "i8_quantize":
        return _case(None, op, _log_int(rng, 1, 4096), 0, _log_int(rng, 1, 11008), dtype, pad=pad)
    act, bias = (rng.choice(["none", "gelu"]), rng.random() < 0.5) if op.startswith("i8") else ("none", False)
    if op == "i8_linear":
        T, R, K = _log_int(rng, 1, 2048), _log_int(rng, 64, 11008), _log_int(rng, 64, 4096)
        E = rest = 0
    else:
        E = _log_int(rng, 1, 64)
        T, R = _log_int(rng, 1, 4096), _log_int(rng, 64, 2048)
        K = _log_int(rng, 64, max(64, min(4096, (1 << 26) // (E * R))))
        rest = rng.choice([0, 0, rng.randint(1, T)])
    return _case(None, op, T, R, max(M, K // M * M), dtype, E=E, N=N, M=M, act=act, pad=pad, bias=bias, rest=rest)


# ---------------------------------------------------------------- inputs
def _inputs(case, seed):
    """Activations ~ N(0, 1) with a few channels ten times as large, weights
    ~ N(0, 0.02) with a size of its own for each channel, gradients ~ N(0,
    0.1); rows go to experts by a router with unequal preferences."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, R, K, E = case["T"], case["R"], case["K"], case["E"]
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    loud = 1.0 + 9.0 * (torch.rand(K, generator=gen, device="cuda") < 0.01)
    wide = torch.zeros(T, K + case["pad"], device="cuda", dtype=dt)
    X = wide[:, :K]
    X.copy_(normal(T, K) * loud)
    d = {"X": X}
    if case["op"] != "i8_quantize":
        lead = (E,) if E else ()
        W = normal(*lead, R, K) * 0.02 * torch.exp(0.3 * normal(*lead, R, 1))
        d["W"] = W.to(dt)
    if case["op"] == "expert_train":
        d["dY"] = (normal(T, R) * 0.1).to(dt)
    if case["bias"]:
        d["bias"] = normal(*((E, R) if E else (R,)))
    if E:
        rows = max(0, T - case["rest"])
        preference = torch.softmax(0.5 * normal(E), 0).cumsum(0)
        preference[-1] = 2.0                              # (the sum may round below one)
        chosen = torch.rand(rows, generator=gen, device="cuda")
        # expert e's rows end where the preferences of those up to e do
        ends = (chosen[:, None] < preference[None, :]).sum(0) if rows else torch.zeros(E, device="cuda")
        d["offsets"] = torch.cat([torch.zeros(1, device="cuda"), ends]).to(torch.int32)
    return d


def _keep(W, N, M):
    """Truth values of the N largest magnitudes of every M along a row, equal
    ones going to the lower position."""
    a = W.float().abs().unflatten(-1, (-1, M))
    keep = torch.empty(a.shape, dtype=torch.bool, device=W.device)
    for i in range(M):
        rank = torch.zeros(a.shape[:-1], dtype=torch.int32, device=W.device)
        for j in range(M):
            if j != i:
                rank += (a[..., j] > a[..., i]) if j > i else (a[..., j] >= a[..., i])
        keep[..., i] = rank < N
    return keep.flatten(-2)


def _i8_round(x):
    """(elements as whole numbers in binary32, scales [..., 1] in binary32) of
    x's rows; the quotient in 64 bits, where none is rounded across a border."""
    s = (x.float().abs().amax(dim=-1, keepdim=True) / 127.0).clamp(min=2.0 ** -126)
    return torch.round(x.double() / s.double()).clamp(-127, 127).float(), s


def prepare(case, seed):
    """The call's operands as a program holds them: activations, offsets, and
    the weights pruned (8 bits: quantised, then pruned) once when the model
    was loaded."""
    d = _inputs(case, seed)
    op, N, M = case["op"], case["N"], case["M"]
    state = {"case": case, **{k: d.get(k) for k in ("X", "dY", "bias", "offsets")}}
    if op == "i8_quantize":
        return state
    W = d["W"]
    if own:
        import semi_structured_sparse_nm_amd as nm
        if op.startswith("i8"):
            q = nm.i8_quantize(W.flatten(0, -2))
            W, state["scale"] = q.values.unflatten(0, W.shape[:-1]), q.scales.unflatten(0, W.shape[:-1])
        state["W"] = nm.pack_experts(W, N, M) if case["E"] else nm.pack(W, N, M)
        return state
    if op.startswith("i8"):
        W, state["scale"] = _i8_round(W)
    state["keep"] = _keep(W, N, M)
    state["W"] = torch.where(state["keep"], W, torch.zeros_like(W))
    if op.startswith("i8"):
        state["W"] = state["W"].to(torch.int8)
    return state


# ---------------------------------------------------------------- plain forms
def _i8_product(x, W, scale, bias, act):
    q, s = _i8_round(x)
    y = (q @ W.float().t()) * s * scale.t()
    if bias is not None:
        y = y + bias
    return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5))) if act == "gelu" else y


def _plain(state):
    case, X = state["case"], state["X"]
    op, act, dt = case["op"], case["act"], X.dtype
    if op == "i8_quantize":
        q, s = _i8_round(X)
        return (q * s).to(dt)
    W, bias = state["W"], state["bias"]
    if op == "i8_linear":
        return _i8_product(X, W, state["scale"], bias, act).to(dt)
    at = state["offsets"].tolist()
    Y = torch.zeros(case["T"], case["R"], device=X.device, dtype=dt)
    dX = torch.zeros(case["T"], case["K"], device=X.device, dtype=dt)
    dW = torch.zeros(W.shape, device=X.device, dtype=dt) if op == "expert_train" else None
    for e in range(case["E"]):
        s = slice(at[e], at[e + 1])
        x = X[s]
        if op == "i8_expert_linear":
            if len(x):
                Y[s] = _i8_product(x, W[e], state["scale"][e], None if bias is None else bias[e], act).to(dt)
            continue
        w = W[e].float()
        Y[s] = (x.float() @ w.t()).to(dt)
        if op == "expert_train":
            dy = state["dY"][s].float()
            dX[s] = (dy @ w).to(dt)
            dW[e] = torch.where(state["keep"][e], dy.t() @ x.float(), 0.0).to(dt)
    return (Y, dX, dW) if op == "expert_train" else Y


def _own(state):
    import semi_structured_sparse_nm_amd as nm
    case, X, W = state["case"], state["X"], state.get("W")
    op = case["op"]
    if op == "i8_quantize":
        return nm.i8_dequantize(nm.i8_quantize(X), out_dtype=X.dtype)
    if op == "i8_linear":
        return nm.i8_linear(W, state["scale"], X, bias=state["bias"], act=case["act"])
    if op == "i8_expert_linear":
        return nm.i8_expert_linear(W, state["scale"], X, state["offsets"], bias=state["bias"], act=case["act"])
    Y = nm.expert_linear(W, X, state["offsets"])
    if op == "expert_linear":
        return Y
    return (Y, *nm.expert_linear_backward(W, X, state["offsets"], state["dY"]))


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: inputs and outputs once, the weights
    in their packed form (of the experts that about that many rows reach),
    products with kept weights only."""
    op, T, R, K, E = case["op"], case["T"], case["R"], case["K"], case["E"]
    N, M = case["N"], case["M"]
    if op == "i8_quantize":
        return {"bytes": 4 * T * K, "flops": 0}
    kept = R * K * N / M
    packed = kept * ((1 if op.startswith("i8") else 2) + (0 if N == M else (2 if M == 4 else 3) / 8))
    packed += 4 * R * (op.startswith("i8") + case["bias"])
    rows = max(0, T - case["rest"])
    reached = E * (1.0 - (1.0 - 1.0 / E) ** rows) if E else 1
    io = 2 * rows * K + 2 * T * R
    if op == "expert_train":
        # forward and both directions of the backward pass: X and dY again in,
        # dX and every expert's weight gradient out
        return {"bytes": io + 2 * rows * R + 2 * T * K + reached * packed + 2 * E * R * K, "flops": 6 * rows * kept}
    return {"bytes": io + reached * packed, "flops": 2 * (rows if E else T) * kept}


# ---------------------------------------------------------------- 64 bits
def _exact_i8(x):
    """(elements, scales) in float64 from the format's definition: the nearest
    whole number of x / scale, the even one where two are equally near, with
    the scale as it is stored."""
    top = x.double().abs().max(dim=-1, keepdim=True).values
    s = (top / 127.0).float().double().clamp(min=2.0 ** -126)
    u = x.double() / s
    low = torch.floor(u)
    up = (u - low > 0.5) | ((u - low == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return torch.minimum(torch.maximum(low + up, u.new_tensor(-127.0)), u.new_tensor(127.0)), s


def _exact_keep(W, N, M):
    order = W.double().abs().unflatten(-1, (-1, M)).sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros(order.shape, dtype=torch.bool, device=W.device)
    keep.scatter_(-1, order[..., :N], True)
    return keep.flatten(-2)


def exact(case, seed):
    d = _inputs(case, seed)
    op, X = case["op"], d["X"]
    if op == "i8_quantize":
        q, s = _exact_i8(X)
        return q * s
    E, T, R, K = case["E"], case["T"], case["R"], case["K"]
    at = d["offsets"].tolist() if E else [0, T]
    Y = torch.zeros(T, R, dtype=torch.float64, device=X.device)
    dX = torch.zeros(T, K, dtype=torch.float64, device=X.device)
    dW = torch.zeros(E, R, K, dtype=torch.float64, device=X.device) if op == "expert_train" else None
    for e in range(max(E, 1)):
        a, b = at[e], at[e + 1]
        w = d["W"][e] if E else d["W"]
        if op.startswith("i8"):
            w, sw = _exact_i8(w)
        keep = _exact_keep(w, case["N"], case["M"])
        w = w.double() * keep
        if b > a and op.startswith("i8"):
            q, sx = _exact_i8(X[a:b])
            y = (q @ w.t()) * (sx * sw.t())
            if "bias" in d:
                y = y + (d["bias"][e] if E else d["bias"]).double()
            Y[a:b] = y * 0.5 * torch.erfc(-y / math.sqrt(2.0)) if case["act"] == "gelu" else y
        elif b > a:
            x = X[a:b].double()
            Y[a:b] = x @ w.t()
            if op == "expert_train":
                dy = d["dY"][a:b].double()
                dX[a:b] = dy @ w
                dW[e] = (dy.t() @ x) * keep
    return (Y, dX, dW) if op == "expert_train" else Y
