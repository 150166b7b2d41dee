"""The dense row operators: linear layers with a fused epilogue and layer norm, forward and backward.

Rows are edges or nodes of a neighbour graph; a row holds C channels. Either the rows lie one after another
([rows, C]), or they are one rank's block of node features [nodes, (lmax + 1)^2, C]: rows l^2 .. (l+1)^2 of each
node, a strided view (l = 0: the node's scalars).

    linear forward     z = x W + bias;  out = act(z) + residual;  with "train" z is returned too
    linear backward    dz = g act'(z);  grad_x = dz W^T;  grad_W = x^T dz;  grad_bias = sum of dz over the rows
    layer norm forward out = (x - mean) rstd weight + bias;  mean and rstd are returned too
    layer norm backward grad_x, grad_weight, grad_bias of the same

All tensors of a call have one type; mean and rstd are float32. act: none, or SiLU(z) = z / (1 + exp(-z)).
"""
import math

import torch

own = False

EPS = 1e-5


def _linear(name, way, rows, k, n, act, dtype="float32", bias=True, residual=False, train=False, lmax=-1, l=0):
    return {"name": name, "op": "linear", "way": way, "rows": rows, "k": k, "n": n, "act": act, "dtype": dtype,
            "bias": bias, "residual": residual, "train": train, "lmax": lmax, "l": l}


def _norm(name, way, rows, k, dtype="float32", lmax=-1, l=0):
    return {"name": name, "op": "norm", "way": way, "rows": rows, "k": k, "dtype": dtype, "lmax": lmax, "l": l}


def listed():
    return [
        # one atom's update while a structure is built up atom by atom: latency alone counts
        _linear("linear one atom", "forward", 1, 128, 128, "silu", residual=True),
        # mixing the channels of the rank-2 features of 4096 nodes, L = 3, C = 128: a strided block, no activation
        _linear("linear rank-2 block", "forward", 4096, 128, 128, "none", bias=False, residual=True, lmax=3, l=2),
        # a scalar-track layer on the edges of the 1024-node, 128-neighbour graph, in training: z is kept
        _linear("linear edges, train", "forward", 131072, 128, 128, "silu", residual=True, train=True),
        # a wider layer on the same edges: as much arithmetic as memory traffic
        _linear("linear edges, 256", "forward", 131072, 256, 256, "silu"),
        # the last layer of the radial weights, P * C = 34 * 128 columns
        _linear("linear radial weights", "forward", 16384, 64, 4352, "none"),
        # a wide layer on the water box's edges in bf16, an odd number of rows
        _linear("linear bf16 wide", "forward", 166517, 256, 512, "silu", dtype="bfloat16"),
        # gradients of a small layer of odd widths (rows that are not 16-byte aligned)
        _linear("linear backward, odd", "backward", 1000, 99, 37, "silu"),
        # gradients of the scalar-track layer on the edges
        _linear("linear backward, edges", "backward", 131072, 128, 128, "silu"),
        # gradients of a wider bf16 layer
        _linear("linear backward, bf16", "backward", 131072, 256, 256, "silu", dtype="bfloat16"),
        # layer norm of the scalars of 1024 nodes, read in place from the features (L = 3, C = 128)
        _norm("norm node scalars", "forward", 1024, 128, lmax=3, l=0),
        # gradients of the layer norm on the edges
        _norm("norm backward, edges", "backward", 131072, 128),
        # the same in bf16 with an odd width
        _norm("norm backward, bf16 odd", "backward", 32768, 515, dtype="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["float32", "float32", "bfloat16"])
    way = rng.choice(["forward", "backward"])
    lmax = rng.choice([-1, -1, 1, 2, 3])
    l = rng.randint(0, lmax) if lmax > 0 else 0
    groups = (lmax + 1) ** 2 if lmax > 0 else 1  # a feature tensor holds every rank's rows
    if rng.random() < 0.65:
        k = _log_int(rng, 4, 512)
        n = _log_int(rng, 4, 512) if rng.random() < 0.85 else _log_int(rng, 512, 4352)
        if rng.random() < 0.5:  # widths of real layers are mostly multiples of 8
            k, n = 8 * max(1, k // 8), 8 * max(1, n // 8)
        most = min(131072, 2**33 // (2 * k * n), 2**26 // (max(k, n) * groups))
        rows = _log_int(rng, 1, max(2, most))
        case = _linear("", way, rows, k, n, rng.choice(["silu", "silu", "none"]), dtype, rng.random() < 0.7,
                       way == "forward" and rng.random() < 0.5, way == "forward" and rng.random() < 0.3, lmax, l)
    else:
        k = _log_int(rng, 4, 2048)
        if rng.random() < 0.5:
            k = 8 * max(1, k // 8)
        rows = _log_int(rng, 1, max(2, min(131072, 2**25 // (k * groups))))
        case = _norm("", way, rows, k, dtype, lmax, l)
    del case["name"]
    return case


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 17)
    dt = getattr(torch, case["dtype"])
    rows, k, l = case["rows"], case["k"], case["l"]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + shift).to(dt)

    def features(c):
        """Rows of c channels: [rows, c], or rank l's block of a feature tensor."""
        if case["lmax"] < 0:
            return normal(rows, c)
        return normal(rows, (case["lmax"] + 1) ** 2, c)[:, l * l:(l + 1) * (l + 1), :]

    st = dict(case)
    if case["op"] == "linear":
        n = case["n"]
        st["x"] = features(k)
        st["W"] = normal(k, n, scale=k ** -0.5)
        st["bias"] = normal(n, scale=0.1) if case["bias"] else None
        if case["way"] == "forward":
            st["residual"] = features(n) if case["residual"] else None
        else:
            st["g"] = features(n)
            st["z"] = None
            if case["act"] == "silu":  # what the forward pass kept
                z = st["x"].float() @ st["W"].float()
                st["z"] = (z + st["bias"].float() if case["bias"] else z).to(dt)
    else:
        x = features(k)
        x.mul_(1.5).add_(0.3)
        st["x"] = x
        st["weight"] = normal(k, scale=0.1, shift=1.0)
        st["bias"] = normal(k, scale=0.1)
        if case["way"] == "backward":
            st["g"] = features(k)
            xf = x.double()  # what the forward pass kept
            mean = xf.mean(-1)
            st["mean"] = mean.float()
            st["rstd"] = ((xf - mean[..., None]).square().mean(-1) + EPS).rsqrt().float()
    return st


def _flat(t):
    """[..., C] as a matrix of rows."""
    return t.reshape(-1, t.shape[-1])


def _plain_linear_forward(st):
    dt = st["x"].dtype
    z = st["x"].float() @ st["W"].float()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    out = z / (1 + torch.exp(-z)) if st["act"] == "silu" else z
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return {"out": out.to(dt), "z": z.to(dt)} if st["train"] else {"out": out.to(dt)}


def _plain_linear_backward(st):
    dt = st["x"].dtype
    dz = st["g"].float()
    if st["act"] == "silu":
        z = st["z"].float()
        s = 1 / (1 + torch.exp(-z))
        dz = dz * (s * (1 + z * (1 - s)))
    grads = {"grad_x": (dz @ st["W"].float().t()).to(dt), "grad_W": (_flat(st["x"].float()).t() @ _flat(dz)).to(dt)}
    if st["bias"] is not None:
        grads["grad_bias"] = _flat(dz).sum(0).to(dt)
    return grads


def _plain_norm_forward(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    out = c * rstd * st["weight"].float() + st["bias"].float()
    return {"out": out.to(st["x"].dtype), "mean": mean[..., 0], "rstd": rstd[..., 0]}


def _plain_norm_backward(st):
    dt = st["x"].dtype
    g = st["g"].float()
    rstd = st["rstd"][..., None]
    xhat = (st["x"].float() - st["mean"][..., None]) * rstd
    gw = g * st["weight"].float()
    gx = rstd * (gw - gw.mean(-1, keepdim=True) - xhat * (gw * xhat).mean(-1, keepdim=True))
    return {"grad_x": gx.to(dt), "grad_weight": _flat(g * xhat).sum(0).to(dt), "grad_bias": _flat(g).sum(0).to(dt)}


def run(st):
    if own:
        import cg_tensor_products_b200 as etp

        if st["op"] == "linear":
            if st["way"] == "forward":
                r = etp.linear_forward(st["x"], st["W"], bias=st["bias"], activation=st["act"],
                                       residual=st["residual"], save_z=st["train"])
                return {"out": r[0], "z": r[1]} if st["train"] else {"out": r}
            gx, gw, gb = etp.linear_backward(st["x"], st["W"], st["g"], z=st["z"], activation=st["act"],
                                             want=("x", "W", "bias") if st["bias"] is not None else ("x", "W"))
            return {"grad_x": gx, "grad_W": gw} if gb is None else {"grad_x": gx, "grad_W": gw, "grad_bias": gb}
        if st["way"] == "forward":
            out, mean, rstd = etp.layer_norm_forward(st["x"], st["weight"], st["bias"], eps=EPS)
            return {"out": out, "mean": mean, "rstd": rstd}
        gx, gw, gb = etp.layer_norm_backward(st["x"], st["weight"], st["mean"], st["rstd"], st["g"])
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if st["op"] == "linear":
        return _plain_linear_forward(st) if st["way"] == "forward" else _plain_linear_backward(st)
    return _plain_norm_forward(st) if st["way"] == "forward" else _plain_norm_backward(st)


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    rows = case["rows"] * (2 * case["l"] + 1)
    k = case["k"]
    if case["op"] == "linear":
        n = case["n"]
        weights = k * n + (n if case["bias"] else 0)
        if case["way"] == "forward":
            per_row = k + n + (n if case["residual"] else 0) + (n if case["train"] else 0)
            return {"bytes": size * (rows * per_row + weights), "flops": 2 * rows * k * n}
        per_row = 2 * k + n + (n if case["act"] == "silu" else 0)  # x, grad_x, g, z
        return {"bytes": size * (rows * per_row + k * n + weights), "flops": 4 * rows * k * n}
    if case["way"] == "forward":
        return {"bytes": size * (2 * rows * k + 2 * k) + 8 * rows, "flops": 8 * rows * k}
    return {"bytes": size * (3 * rows * k + 3 * k) + 8 * rows, "flops": 13 * rows * k}


def exact(case, seed):
    """The definition in 64 bits; gradients by differentiating it."""
    st = prepare(case, seed)

    def wide(key):
        v = st.get(key)
        return None if v is None else v.detach().to(torch.float64)

    if case["op"] == "linear":
        x, W, b = wide("x"), wide("W"), wide("bias")
        if case["way"] == "forward":
            z = torch.einsum("...k,kn->...n", x, W)
            z = z if b is None else z + b
            a = 0.5 * z * (1 + torch.tanh(0.5 * z)) if case["act"] == "silu" else z
            r = wide("residual")
            out = a if r is None else a + r
            return {"out": out, "z": z} if case["train"] else {"out": out}
        dz = wide("g")
        if case["act"] == "silu":  # at the kept z, which is an input here
            z = wide("z").requires_grad_()
            (dz,) = torch.autograd.grad(0.5 * z * (1 + torch.tanh(0.5 * z)), z, dz)
        grads = {"grad_x": torch.einsum("...n,kn->...k", dz, W)}
        grads["grad_W"] = torch.einsum("rk,rn->kn", _flat(x), _flat(dz))
        if b is not None:
            grads["grad_bias"] = torch.einsum("rn->n", _flat(dz))
        return grads
    x, w, b = wide("x").requires_grad_(), wide("weight").requires_grad_(), wide("bias").requires_grad_()
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    rstd = (var + EPS) ** -0.5
    out = (x - mean) * rstd * w + b
    if case["way"] == "forward":
        return {"out": out.detach(), "mean": mean.detach()[..., 0], "rstd": rstd.detach()[..., 0]}
    gx, gw, gb = torch.autograd.grad(out, (x, w, b), wide("g"))
    return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
