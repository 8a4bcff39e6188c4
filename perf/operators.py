"""Cases of the routing and int8 expert operators, with their plain forms and 64-bit references.

Operators
  route     scores (softmax or sigmoid) + balance bias + expert groups + top-k + weights
  quantize  int8 codes and one scale per row
  linear    grouped product of int8 rows with each group's int8 matrix, scales per row and output channel
  ffn       grouped SwiGLU expert FFN on int8 weights and int8 activations

Sizes are those of the repository's workloads (64 experts top-8 at 2048 x 1024, 64 + 2 shared experts top-6 at
2048 x 1408, 128 experts top-8 at 2048 x 768, 128 experts top-4 at 2880 x 2880) and ragged ones between them.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128          # columns of the SwiGLU product that share one scale


def listed():
    return [
        # --- route: one decode step of a small batch; a prompt on a grouped sigmoid router; a ragged softmax batch in bf16
        dict(name="route_decode", op="route", T=16, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             rank="top2", renorm=True, scale=2.5, dtype="f32"),
        dict(name="route_prompt", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             rank="top2", renorm=True, scale=2.5, dtype="f32"),
        dict(name="route_ragged_bf16", op="route", T=4159, E=160, k=6, score="softmax", bias=False, groups=8,
             top_groups=3, rank="max", renorm=False, scale=1.0, dtype="bf16"),
        # --- quantize: the rows of a decode step, and of a prompt of odd length
        dict(name="quantize_decode", op="quantize", T=128, d=2048, dtype="bf16"),
        dict(name="quantize_prompt", op="quantize", T=8191, d=2880, dtype="bf16"),
        # --- linear: one dense projection of a few tokens; the experts' up projection in a decode step; a dense
        #     projection of a prompt, fp32 out
        dict(name="linear_few", op="linear", T=5, E=1, k=1, K=2048, O=2048, zipf=0.0, out="bf16"),
        dict(name="linear_experts_decode", op="linear", T=128, E=64, k=8, K=2048, O=1024, zipf=0.5, out="bf16"),
        dict(name="linear_prompt", op="linear", T=8191, E=1, k=1, K=2048, O=4096, zipf=0.0, out="f32"),
        # --- ffn: a single token; a decode step with two shared experts and hot ones; a prompt; decode tokens ahead of a
        #     prefill chunk (a priority segment) on the widest experts
        dict(name="ffn_one_token", op="ffn", T=1, E=64, k=8, S=0, prio=0, d=2048, I=1024, zipf=0.5),
        dict(name="ffn_decode_shared", op="ffn", T=77, E=64, k=6, S=2, prio=0, d=2048, I=1408, zipf=1.1),
        dict(name="ffn_prompt", op="ffn", T=4096, E=128, k=8, S=0, prio=0, d=2048, I=768, zipf=0.3),
        dict(name="ffn_mixed", op="ffn", T=1088, E=128, k=4, S=0, prio=64, d=2880, I=2880, zipf=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "linear", "ffn", "ffn"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(3, 512 // groups if groups > 1 else 400)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(16, top * (E // groups)))
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.6, groups=groups, top_groups=top, rank=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 8192), d=8 * _log(rng, 4, 360), dtype=rng.choice(["f32", "bf16"]))
    if op == "linear":
        E = rng.choice([1, 1, 8, 64, 128])
        k = 1 if E == 1 else rng.choice([2, 4, 8])
        return dict(op=op, T=_log(rng, 1, 4096 if E == 1 else 1024), E=E, k=k, K=64 * rng.randint(2, 40),
                    O=64 * rng.randint(2, 40), zipf=0.0 if E == 1 else rng.choice([0.0, 0.5, 1.0]),
                    out=rng.choice(["f32", "bf16"]))
    E = rng.choice([8, 16, 64, 128])
    k, S, d, I = rng.choice([1, 2, 4, 8]), rng.choice([0, 0, 1, 2]), 64 * rng.randint(2, 40), 64 * rng.randint(2, 24)
    T = min(_log(rng, 1, 2048), int(5e10 / (d * I * (k + S))))
    return dict(op=op, T=T, E=E, k=k, S=S, prio=rng.choice([0, 0, min(T, rng.randint(1, 64))]), d=d, I=I,
                zipf=rng.choice([0.0, 0.5, 1.0]))


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _weights(g, n, rows, cols):
    """n matrices [rows][cols] of N(0, 0.02^2) weights as int8 codes and a scale per row (amax / 127)."""
    q = torch.empty((n, rows, cols), dtype=torch.int8, device=DEV)
    s = torch.empty((n, rows), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (rows * cols))
    for a in range(0, n, step):
        w = torch.randn((min(step, n - a), rows, cols), generator=g, device=DEV).mul_(0.02)
        m = w.abs().amax(-1) / 127.0
        s[a:a + step] = m
        q[a:a + step] = (w / m.unsqueeze(-1)).round_().to(torch.int8)
    return q, s


def _packed(q):
    """The layout that the kernels read: blocks of 16 rows x 64 codes, (row block, column block) order; inside a block the
    16 codes of columns 16 j .. 16 j + 15 of row r at byte (16 j + r) * 16."""
    n, rows, cols = q.shape
    return q.view(n, rows // 16, 16, cols // 64, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous().view(n, rows, cols)


def _rows(g, T, d, dtype):
    """Hidden states: N(0, 1) with token-dependent size and a few large channels."""
    x = torch.randn((T, d), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV))
    x[:, torch.randint(0, d, (max(1, d // 256),), generator=g, device=DEV)] *= 8.0
    return x.to(dtype)


def _plan(g, T, E, k, S, prio, zipf):
    """The batch's dispatch: sorted rows grouped by (segment, expert), then the shared experts; the row list and the
    group offsets that moe_permute makes.  Also the rows of the fullest expert, which a program that pads keeps."""
    l = torch.randn((T, E), generator=g, device=DEV)
    l -= zipf * torch.log1p(torch.randperm(E, generator=g, device=DEV).float())
    ids = l.topk(min(k, E), dim=1).indices
    seg = torch.zeros(T, dtype=torch.int64, device=DEV)
    nseg = 2 if prio > 0 else 1
    if prio > 0:
        seg[prio:] = 1
    group = (seg[:, None] * E + ids).reshape(-1)
    tok = torch.arange(T, device=DEV)
    token = tok.repeat_interleave(ids.shape[1])
    if S:
        group = torch.cat([group, nseg * E + torch.arange(S, device=DEV).repeat_interleave(T)])
        token = torch.cat([token, tok.repeat(S)])
    order = torch.argsort(group, stable=True)
    G = nseg * E + S
    counts = torch.bincount(group, minlength=G)
    offs = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    offs[1:] = counts.cumsum(0)
    routed = counts[:nseg * E].view(nseg, E).sum(0)
    return dict(x_rows=token[order].to(torch.int32), offs=offs, nseg=nseg, cap=int(torch.cat([routed, counts[nseg * E:]]).max()))


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = torch.randn((T, E), generator=g, device=DEV).mul_(1.5).to(_dt(case["dtype"]))
        st["bias"] = torch.randn((E,), generator=g, device=DEV).mul_(0.05) if case["bias"] else None
        st["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        st["w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    elif op == "quantize":
        T, d = case["T"], case["d"]
        st["x"] = _rows(g, T, d, _dt(case["dtype"]))
        st["q"] = torch.empty((T, d), dtype=torch.int8, device=DEV)
        st["s"] = torch.empty((T,), dtype=torch.float32, device=DEV)
    elif op == "linear":
        K, O, E = case["K"], case["O"], case["E"]
        st.update(_plan(g, case["T"], E, case["k"], 0, 0, case["zipf"]))
        x = _rows(g, case["T"], K, torch.float32)
        st["xs"] = x.abs().amax(1) / 127.0
        st["xq"] = (x / st["xs"][:, None]).round().to(torch.int8)
        st["w"], st["sw"] = _weights(g, E, O, K)
        st["w_packed"] = _packed(st["w"])
        st["y"] = torch.empty((st["x_rows"].numel(), O), dtype=_dt(case["out"]), device=DEV)
    else:
        d, I, n = case["d"], case["I"], case["E"] + case["S"]
        st.update(_plan(g, case["T"], case["E"], case["k"], case["S"], case["prio"], case["zipf"]))
        st["x"] = _rows(g, case["T"], d, torch.bfloat16)
        for name, rows, cols in (("gate", I, d), ("up", I, d), ("down", d, I)):
            q, s = _weights(g, n, rows, cols)
            st["q_" + name], st["s_" + name], st["p_" + name] = q, s, _packed(q)
        N = st["x_rows"].numel()
        st["h"] = torch.empty((N, d), dtype=torch.bfloat16, device=DEV)
        # the call's scratch: int8 tokens and their scales, the int8 SwiGLU product and its block scales
        st["ws"] = torch.empty(case["T"] * (d + 16) + N * (I + 4 * (I // BLOCK + 1)) + 65536, dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------------------------------- plain forms
def _plain_route(st, c):
    E, k, ng = c["E"], c["k"], c["groups"]
    l = st["logits"].double()
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    choice = l if st["bias"] is None else s + st["bias"].double()
    if ng > 1:
        v = (s if st["bias"] is None else choice).view(-1, ng, E // ng)
        if c["rank"] == "max":
            v = choice.view(-1, ng, E // ng).amax(2)
        else:
            v = v.topk(min(2, E // ng), dim=2).values.sum(2)
        best = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(v, dtype=torch.bool).scatter_(1, best, True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // ng, 1), -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_quantize(x, block=None):
    """Codes (as floats) and scales of the rows, or of each `block` columns of a row.  The quotient is taken in 64 bits:
    next to a border between two codes a 32-bit one falls on the wrong side."""
    v = x if block is None else torch.nn.functional.pad(x, (0, -x.shape[-1] % block)).unflatten(-1, (-1, block))
    v = v.float()
    s = v.abs().amax(-1) / 127.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (v.double() / s.double().unsqueeze(-1)).round().clamp(-127, 127).float()
    return q, s


def _slots(st, E, S):
    """Rows of the experts (an expert's rows of both segments together), padded to the largest: [E+S][cap] sorted row
    numbers and which of them exist."""
    offs, nseg = st["offs"].long(), st["nseg"]
    row = torch.arange(st["x_rows"].numel(), device=DEV)
    g = torch.searchsorted(offs[1:], row, right=True)
    e = torch.where(g < nseg * E, g % E, g - (nseg - 1) * E)
    order = torch.argsort(e, stable=True)
    ends = torch.searchsorted(e[order], torch.arange(E + S, device=DEV), right=True)
    at = torch.cat([ends.new_zeros(1), ends[:-1]])[:, None] + torch.arange(st["cap"], device=DEV)
    there = at < ends[:, None]
    return order[torch.where(there, at, 0)], there


def _plain_linear(st, c):
    at, there = _slots(st, c["E"], 0)
    rows = st["x_rows"].long()[at]                                                     # [E][cap] tokens
    x = st["xq"][rows].float()
    v = torch.bmm(st["w"].float(), x.transpose(1, 2).contiguous()).transpose(1, 2)     # [E][cap][O]
    v = v * st["xs"][rows].unsqueeze(-1) * st["sw"].unsqueeze(1)
    y = torch.empty_like(st["y"])
    y[at[there]] = v[there].to(y.dtype)
    return y


def _plain_ffn(st, c):
    at, there = _slots(st, c["E"], c["S"])
    rows = st["x_rows"].long()[at]
    xq, xs = _plain_quantize(st["x"])
    x = xq[rows].transpose(1, 2).contiguous()                                          # [E+S][d][cap]
    sx = xs[rows].unsqueeze(-1)
    g = torch.bmm(st["q_gate"].float(), x).transpose(1, 2) * sx * st["s_gate"].unsqueeze(1)
    u = torch.bmm(st["q_up"].float(), x).transpose(1, 2) * sx * st["s_up"].unsqueeze(1)
    aq, sa = _plain_quantize(g / (1.0 + torch.exp(-g)) * u, BLOCK)                     # [E+S][cap][blocks][128], its scales
    a = (aq * sa.unsqueeze(-1)).flatten(2)[..., :c["I"]]
    v = torch.bmm(st["q_down"].float(), a.transpose(1, 2).contiguous()).transpose(1, 2) * st["s_down"].unsqueeze(1)
    h = torch.empty_like(st["h"])
    h[at[there]] = v[there].to(h.dtype)
    return h


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import top_expert_routing_amd as moe
        if op == "route":
            return moe.route(st["logits"], c["k"], score=c["score"], bias=st["bias"], n_groups=c["groups"],
                             top_groups=c["top_groups"], group_rank=c["rank"], renormalize=c["renorm"],
                             scale=c["scale"], topk_ids=st["ids"], topk_w=st["w"])
        if op == "quantize":
            q, s = moe.quantize_rows_i8(st["x"], st["q"], st["s"])
            return q, s
        if op == "linear":
            return moe.grouped_linear_i8(st["xq"], st["xs"], st["offs"], c["E"], 0, st["nseg"], st["w_packed"], st["sw"],
                                         st["y"], x_rows=st["x_rows"])
        return moe.grouped_ffn_i8(st["x"], st["offs"], c["E"], c["S"], st["nseg"], st["p_gate"], st["s_gate"],
                                  st["p_up"], st["s_up"], st["p_down"], st["s_down"], st["h"], st["ws"],
                                  x_rows=st["x_rows"])
    if op == "route":
        return _plain_route(st, c)
    if op == "quantize":                   # the codes are whole numbers by an exact rule, so they come back as they are
        q, s = _plain_quantize(st["x"])
        return q.to(torch.int8), s
    if op == "linear":
        return _plain_linear(st, c)
    return _plain_ffn(st, c)


# ---------------------------------------------------------------------------------------------------- work
def _used(c, n):
    """Experts that n rows reach, if they were spread evenly: at most the rows, at most all."""
    return min(c["E"], n)


def work(case):
    c = case
    if c["op"] == "route":
        es = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["T"] * c["E"] * es + c["T"] * c["k"] * 8 + 4 * c["E"] * c["bias"], flops=10.0 * c["T"] * c["E"])
    if c["op"] == "quantize":
        es = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["T"] * (c["d"] * (es + 1) + 4), flops=5.0 * c["T"] * c["d"])
    if c["op"] == "linear":
        k = min(c["k"], c["E"])
        N = c["T"] * k
        es = 4 if c["out"] == "f32" else 2
        return dict(bytes=_used(c, N) * c["O"] * (c["K"] + 4) + c["T"] * (c["K"] + 4) + N * (c["O"] * es + 4),
                    flops=2.0 * N * c["K"] * c["O"])
    k = min(c["k"], c["E"])
    N = c["T"] * (k + c["S"])
    experts = _used(c, c["T"] * k) + c["S"]
    return dict(bytes=experts * (3 * c["d"] * c["I"] + 4 * (2 * c["I"] + c["d"])) + c["T"] * c["d"] * 2 + N * (c["d"] * 2 + 4),
                flops=6.0 * N * c["d"] * c["I"])


# ---------------------------------------------------------------------------------------------------- 64-bit references
def _codes64(v):
    """int8 codes and the fp32 scale of the last axis, by the definition: scale = the largest magnitude / 127 rounded to
    32 bits, code = the nearest integer to value / scale (halves to even)."""
    s = (v.abs().max(-1).values.float() / 127.0).double()
    s[s == 0] = 1.0
    return torch.round(v / s[..., None]).clamp_(-127, 127), s


def _dot_codes(a, w):
    """Sums of products of integer codes, exact: pieces of at most 1024 columns stay below 2^24 in 32 bits
    (1024 * 127 * 127 < 2^24), and the pieces are added in 64."""
    out = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    for i in range(0, a.shape[1], 1024):
        out += (a[:, i:i + 1024].float() @ w[:, i:i + 1024].float().T.contiguous()).double()
    return out


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "route":
        l = st["logits"].cpu().double()
        if c["score"] == "sigmoid":
            s = 1.0 / (1.0 + torch.exp(-l))
        else:
            z = torch.exp(l - l.max(1, keepdim=True).values)
            s = z / z.sum(1, keepdim=True)
        b = torch.zeros(c["E"], dtype=torch.float64) if st["bias"] is None else st["bias"].cpu().double()
        order = (l if st["bias"] is None else s + b).numpy()
        val = (s + b).numpy()
        T, E, k, ng = c["T"], c["E"], c["k"], c["groups"]
        import numpy as np
        if ng > 1:
            size = E // ng
            gv = np.sort((order if c["rank"] == "max" else val).reshape(T, ng, size), axis=2)
            gv = gv[:, :, -1] if c["rank"] == "max" or size == 1 else gv[:, :, -1] + gv[:, :, -2]
            place = np.argsort(np.argsort(-gv, axis=1, kind="stable"), axis=1, kind="stable")
            order = np.where(np.repeat(place < c["top_groups"], size, axis=1), order, -np.inf)
        ids = np.argsort(-order, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(s.numpy(), ids, 1)
        if c["renorm"]:
            w = w / w.sum(1, keepdims=True)
        return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w * c["scale"])
    if c["op"] == "quantize":
        q, s = _codes64(st["x"].double())
        return q.to(torch.int8), s
    offs = st["offs"].tolist()
    rows = st["x_rows"].long()
    if c["op"] == "linear":
        y = torch.empty((rows.numel(), c["O"]), dtype=torch.float64, device=DEV)
        for g in range(c["E"]):
            r = rows[offs[g]:offs[g + 1]]
            if r.numel():
                y[offs[g]:offs[g + 1]] = _dot_codes(st["xq"][r], st["w"][g]) * st["xs"][r].double()[:, None] * st["sw"][g].double()
        return y
    E, nseg, I = c["E"], st["nseg"], c["I"]
    xq, xs = _codes64(st["x"].double())
    h = torch.empty((rows.numel(), c["d"]), dtype=torch.float64, device=DEV)
    for g in range(len(offs) - 1):
        r = rows[offs[g]:offs[g + 1]]
        if not r.numel():
            continue
        e = g % E if g < nseg * E else g - (nseg - 1) * E
        gate = _dot_codes(xq[r], st["q_gate"][e]) * xs[r, None] * st["s_gate"][e].double()
        up = _dot_codes(xq[r], st["q_up"][e]) * xs[r, None] * st["s_up"][e].double()
        a = gate * torch.sigmoid(gate) * up
        acc = torch.zeros((r.numel(), c["d"]), dtype=torch.float64, device=DEV)
        for b in range(0, I, BLOCK):
            q, s = _codes64(a[:, b:b + BLOCK])
            acc += _dot_codes(q, st["q_down"][e][:, b:b + BLOCK]) * s[:, None]
        h[offs[g]:offs[g + 1]] = acc * st["s_down"][e].double()
    return h
