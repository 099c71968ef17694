"""Cases of the training operators, for timing them and comparing them with plain forms.

Three operators finish a training step that starts from event ids:

  tokenwise  the backward pass of the token-wise normalised sketch attention (attention of k
             shared prototypes over each user's events, the probabilities recomputed);
  events     the backward pass of the event rows x_i = item[id_i] + action[a_i], into the two
             embedding tables;
  adamw      the AdamW step over many tensors at once, its states in 32 bits or in 8.

``run`` computes them in elementary torch operations, or, where ``own`` is true, by this
repository's entry points.
"""
import math

import torch

own = False

D = 128          # row width of the events and the prototypes
BLOCK = 128      # values that share one scale of an 8-bit state
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -9
SCALE_MIN = 2.0 ** -100
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.01


def weight_sizes(k, refine, stca):
    """Values of each weight tensor of a model: prototypes and projections (k x 128, three of
    128 x 128), `refine` refinement layers and `stca` full attention layers of 4 heads of 32."""
    sizes = [k * D] + [D * D] * 3
    sizes += ([D * D] * 2 + [D] * 4 + [D * 2 * D] * 3) * refine
    sizes += ([D * D] * 4 + [D * 2 * D] * 6) * stca
    return ",".join(str(s) for s in sizes)


def listed():
    return [
        # one user's short history and few prototypes: a call's fixed cost
        {"name": "tokenwise one short user", "op": "tokenwise", "k": 64, "lens": "300", "scale": 1.0},
        # ragged users with none, one and a tile's edge of events, prototypes that fill no tile
        {"name": "tokenwise ragged odd", "op": "tokenwise", "k": 200, "lens": "0,1,129,2500,1777,128,999", "scale": 2.0},
        # a batch of recent suffixes (10K events each) at half the production prototypes
        {"name": "tokenwise recent suffixes", "op": "tokenwise", "k": 512, "lens": "10000,9000,10000,7321", "scale": 1.0},
        # whole histories (85K events on average, at most 100K) at the production width
        {"name": "tokenwise whole histories", "op": "tokenwise", "k": 1024, "lens": "100000,85000,71234,83777", "scale": 1.0},
        # the events of one short user, a small vocabulary
        {"name": "events one short user", "op": "events", "n": 300, "vocab": 4096, "actions": 8, "dtype": "bf16"},
        # an odd batch
        {"name": "events odd batch", "op": "events", "n": 77777, "vocab": 100003, "actions": 5, "dtype": "bf16"},
        # the refinement's gradient of the event rows comes in 32 bits
        {"name": "events of the refinement", "op": "events", "n": 200000, "vocab": 250000, "actions": 16, "dtype": "f32"},
        # eight users' whole histories against the benchmark's vocabulary
        {"name": "events training step", "op": "events", "n": 680000, "vocab": 1000000, "actions": 8, "dtype": "bf16"},
        # the weights of a sketch model: many small tensors, states in 32 bits and in 8
        {"name": "adamw weights 32", "op": "adamw", "sizes": weight_sizes(1024, 2, 4), "bits": 32, "grad": "f32", "copy": False},
        {"name": "adamw weights 8", "op": "adamw", "sizes": weight_sizes(1024, 2, 4), "bits": 8, "grad": "f32", "copy": False},
        # the item table of the benchmark's vocabulary, with the bf16 copy that the gather reads
        {"name": "adamw table 32", "op": "adamw", "sizes": "128000000", "bits": 32, "grad": "f32", "copy": True},
        {"name": "adamw table 8", "op": "adamw", "sizes": "128000000", "bits": 8, "grad": "f32", "copy": True},
    ]


def spread(rng, low, high):
    """An odd or even whole number, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("tokenwise", "events", "adamw"))
    if op == "tokenwise":
        k = spread(rng, 1, 1024)
        users = rng.randint(1, 6)
        longest = spread(rng, 1, 340000 // users if users > 3 else 100000)
        lens = [longest] + [rng.randint(longest // 2, longest) for _ in range(users - 1)]
        if users > 2 and rng.random() < 0.3:
            lens[rng.randrange(1, users)] = rng.choice((0, 1))
        rng.shuffle(lens)
        return {"op": op, "k": k, "lens": ",".join(str(n) for n in lens), "scale": rng.choice((0.25, 1.0, 2.0))}
    if op == "events":
        return {"op": op, "n": spread(rng, 1, 680000), "vocab": spread(rng, 1, 1000000), "actions": rng.randint(1, 16),
                "dtype": rng.choice(("bf16", "f32"))}
    count = spread(rng, 1, 80)
    sizes = [spread(rng, 1, 128000000 // count) for _ in range(count)]
    return {"op": op, "sizes": ",".join(str(s) for s in sizes), "bits": rng.choice((8, 32)),
            "grad": rng.choice(("f32", "bf16")), "copy": rng.random() < 0.5}


def lengths(text):
    return [int(t) for t in text.split(",")]


def gauss(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"tokenwise": prepare_tokenwise, "events": prepare_events, "adamw": prepare_adamw}[case["op"]](case, gen)


def prepare_tokenwise(case, gen):
    lens, k = lengths(case["lens"]), case["k"]
    offsets = torch.tensor([0] + lens).cumsum(0)
    s = {"op": "tokenwise", "k": k, "longest": max(lens), "eps": 1e-6,
         "offsets": offsets.numpy(), "offsets_dev": offsets.cuda()}
    s["X"] = gauss(gen, sum(lens), D).bfloat16()
    s["P"] = gauss(gen, k, D, std=case["scale"])
    for w in ("W_Q", "W_K", "W_V"):
        s[w] = gauss(gen, D, D, std=D ** -0.5)
    s["dS"] = gauss(gen, len(lens), k, D)
    # H = A X of the forward pass, which a training program keeps for the backward pass
    X, there = padded(s)
    A = probabilities(s, X, there)[0]
    s["H"] = torch.matmul(A, X).contiguous()
    return s


def prepare_events(case, gen):
    n, vocab = case["n"], case["vocab"]
    # item ids by popularity (density ~ rank^-1.1, as the benchmark's events), shuffled over the vocabulary
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = ((1 - u * (1 - (vocab + 1.0) ** -0.1)) ** -10.0 - 1).long().clamp_(0, vocab - 1)
    order = torch.randperm(vocab, generator=gen, device="cuda")
    dX = gauss(gen, n, D)
    return {"op": "events", "vocab": vocab, "actions": case["actions"], "ids": order[rank].int(),
            "acts": torch.randint(0, case["actions"], (n,), generator=gen, device="cuda").to(torch.uint8),
            "dX": dX.bfloat16() if case["dtype"] == "bf16" else dX}


def prepare_adamw(case, gen):
    # the tensors lie in flat buffers, each at a multiple of BLOCK values, as a trainer that
    # reduces its gradients in buckets lays them out
    sizes = lengths(case["sizes"])
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    starts = [0]
    for r in room:
        starts.append(starts[-1] + r)
    total = starts[-1]
    s = {"op": "adamw", "bits": case["bits"], "step": 10, "sizes": sizes, "starts": starts[:-1]}
    s["param"] = gauss(gen, total, std=0.02)
    grad = gauss(gen, total, std=1e-3)
    m = gauss(gen, total, std=1e-3)
    v = gauss(gen, total, std=1e-3).square_()
    for n, r, b in zip(sizes, room, starts):
        for t in (s["param"], grad, m, v):
            t[b + n:b + r] = 0
    s["grad"] = grad.bfloat16() if case["grad"] == "bf16" else grad
    # biases and gains (one row or less) are not decayed
    decay = [DECAY if n > D else 0.0 for n in sizes]
    s["decay"], s["ends"] = torch.tensor(decay, device="cuda"), torch.tensor(starts[1:], device="cuda")
    s["copy"] = s["param"].bfloat16() if case["copy"] else None
    if case["bits"] == 8:
        s["m"], s["m_scale"] = to_8(m)
        s["v"], s["v_scale"] = to_8(v.sqrt_(), floor=True)
    else:
        s["m"], s["v"] = m, v
    if own:
        # the list of tensors that a training program makes once
        import sketch_attention_b200 as sab
        part = lambda name, b, n: None if s.get(name) is None else s[name][b:b + n]  # noqa: E731
        scale = lambda name, b, n: s[name][b // BLOCK:-(-(b + n) // BLOCK)] if case["bits"] == 8 else None  # noqa: E731
        s["tensors"] = sab.AdamWTensors(
            [{"param": part("param", b, n), "grad": part("grad", b, n), "m": part("m", b, n), "v": part("v", b, n),
              "m_scale": scale("m_scale", b, n), "v_scale": scale("v_scale", b, n),
              "param_bf16": part("copy", b, n), "weight_decay": w}
             for b, n, w in zip(s["starts"], sizes, decay)])
    return s


def run(s):
    if own:
        import sketch_attention_b200 as sab
        if s["op"] == "tokenwise":
            return sab.sa_backward_tokenwise(s["X"], s["offsets"], s["P"], s["W_Q"], s["W_K"], s["W_V"], s["eps"],
                                             s["H"], s["dS"], offsets_dev=s["offsets_dev"])
        if s["op"] == "events":
            return sab.sa_gather_events_backward(s["ids"], s["acts"], s["dX"], s["vocab"], s["actions"])
        s["step"] += 1
        sab.sa_adamw_step(s["tensors"], LR, BETA1, BETA2, EPS, step=s["step"])
        return updated(s)
    return {"tokenwise": plain_tokenwise, "events": plain_events, "adamw": plain_adamw}[s["op"]](s)


def updated(s):
    """The buffers that an AdamW step changes."""
    return {name: s[name] for name in ("param", "m", "v", "m_scale", "v_scale", "copy") if s.get(name) is not None}


# ------------------------------------------------------------------ plain forms
def padded(s):
    """The users' events as [users, longest, D] in 32 bits, and which of them are there."""
    off = s["offsets_dev"]
    at = off[:-1, None] + torch.arange(max(s["longest"], 1), device="cuda")
    there = at < off[1:, None]
    return s["X"].float()[at.clamp_max(max(len(s["X"]) - 1, 0))] * there[..., None], there


def probabilities(s, X, there):
    """The token-wise probabilities [users, k, longest] and the folded prototypes."""
    U = s["P"] @ s["W_Q"] @ s["W_K"].T / math.sqrt(D)
    Z = torch.matmul(U, X.transpose(1, 2)).masked_fill_(~there[:, None], -3e38)
    A = (Z - Z.amax(-1, keepdim=True)).exp_() * there[:, None]
    return A.div_(A.sum(-1, keepdim=True).clamp_min_(1e-30)), U


def plain_tokenwise(s):
    X, there = padded(s)
    A, U = probabilities(s, X, there)
    full = there.any(-1)[:, None, None]
    inv = full / (full + s["eps"])
    dH = s["dS"] @ s["W_V"].T * inv
    dZ = (torch.matmul(dH, X.transpose(1, 2)) - (dH * s["H"]).sum(-1, keepdim=True)).mul_(A)
    dX = torch.matmul(A.transpose(1, 2), dH) + torch.matmul(dZ.transpose(1, 2), U)
    E = torch.matmul(dZ, X).sum(0)
    PQ, EK = s["P"] @ s["W_Q"] / math.sqrt(D), E @ s["W_K"] / math.sqrt(D)
    row = torch.arange(len(s["X"]), device="cuda")
    user = torch.searchsorted(s["offsets_dev"], row, right=True) - 1
    return {"dX": dX[user, row - s["offsets_dev"][user]].bfloat16(), "dP": EK @ s["W_Q"].T, "dW_Q": s["P"].T @ EK,
            "dW_K": E.T @ PQ, "dW_V": ((s["H"] * inv).reshape(-1, D).T @ s["dS"].reshape(-1, D))}


def plain_events(s):
    rows, vocab, actions = s["dX"].float(), s["vocab"], s["actions"]
    ids, acts = s["ids"].long(), s["acts"].long()
    there = (ids >= 0) & (ids < vocab) & (acts < actions)
    item = torch.zeros(vocab + 1, D, device="cuda").index_add_(0, torch.where(there, ids, vocab), rows)
    which = (acts[None] == torch.arange(actions, device="cuda")[:, None]) & there
    return {"d_item": item[:vocab], "d_action": which.float() @ rows}


def to_8(x, floor=False):
    """x in e4m3 with one scale for each BLOCK values; with `floor` (x >= 0) no positive value becomes zero."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top >= SCALE_MIN, top / E4M3_MAX, 0.0)
    y = x / torch.where(scale > 0, scale, 1.0) * (scale > 0)
    if floor:
        y = torch.where((x > 0) & (scale > 0), y.clamp_min(E4M3_TINY), y)
    return y.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def plain_adamw(s):
    s["step"] += 1
    g = s["grad"].float()
    if s["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).square_().view(-1)
    else:
        m, v = s["m"], s["v"]
    m = m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v = v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    tensor = torch.searchsorted(s["ends"], torch.arange(0, len(g), BLOCK, device="cuda"), right=True)
    keep = (1 - LR * s["decay"])[tensor, None]
    change = m / (v.sqrt().div_(math.sqrt(1 - BETA2 ** s["step"])).add_(EPS))
    s["param"].view(-1, BLOCK).mul_(keep)
    s["param"].add_(change, alpha=-LR / (1 - BETA1 ** s["step"]))
    if s["copy"] is not None:
        s["copy"].copy_(s["param"])
    if s["bits"] == 8:
        for name, (codes, scale) in (("m", to_8(m)), ("v", to_8(v.sqrt(), floor=True))):
            s[name].copy_(codes)
            s[name + "_scale"].copy_(scale)
    return updated(s)


# ------------------------------------------------------------------ sizes and 64-bit values
def work(case):
    if case["op"] == "tokenwise":
        lens, k = lengths(case["lens"]), case["k"]
        n, B = sum(lens), len(lens)
        # X, H and dS read, dX written, weights read and their gradients written;
        # Z, dA, dZ X, A^T dH and dZ^T U are products of 2 k D a token, the projections 2 D D a row
        return {"bytes": 2 * 2 * n * D + 2 * 4 * B * k * D + 2 * 4 * (k * D + 3 * D * D),
                "flops": 5 * 2.0 * k * D * n + 2.0 * D * D * k * (2 * B + 4)}
    if case["op"] == "events":
        n = case["n"]
        return {"bytes": n * D * (2 if case["dtype"] == "bf16" else 4) + 5 * n + 4 * D * (case["vocab"] + case["actions"]),
                "flops": 2.0 * n * D}
    n = sum(lengths(case["sizes"]))
    per = 8 + (4 if case["grad"] == "f32" else 2) + (2 if case["copy"] else 0)
    per += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * per, "flops": 16.0 * n}


def exact(case, seed):
    with torch.no_grad():
        return {"tokenwise": exact_tokenwise, "events": exact_events, "adamw": exact_adamw}[case["op"]](prepare(case, seed))


def exact_tokenwise(s):
    P, WQ, WK, WV, H, dS = (s[n].double() for n in ("P", "W_Q", "W_K", "W_V", "H", "dS"))
    root = math.sqrt(D)
    U = torch.linalg.multi_dot((P, WQ, WK.T)) / root
    E, dWV, dX = torch.zeros_like(P), torch.zeros_like(WV), []
    for u, (b, e) in enumerate(zip(s["offsets"][:-1].tolist(), s["offsets"][1:].tolist())):
        if b == e:
            continue
        x = s["X"][b:e].double()
        A = torch.softmax(U @ x.T, dim=1)
        dH = dS[u] @ WV.T / (1 + s["eps"])
        dWV += (H[u] / (1 + s["eps"])).T @ dS[u]
        dZ = A * (dH @ x.T - (dH * H[u]).sum(1, keepdim=True))
        E += dZ @ x
        dX.append(A.T @ dH + dZ.T @ U)
    return {"dX": torch.cat(dX) if dX else s["X"].double(), "dP": torch.linalg.multi_dot((E, WK, WQ.T)) / root,
            "dW_Q": torch.linalg.multi_dot((P.T, E, WK)) / root,
            "dW_K": torch.linalg.multi_dot((E.T, P, WQ)) / root, "dW_V": dWV}


def exact_events(s):
    ids, acts, rows = s["ids"].long(), s["acts"].long(), s["dX"].double()
    keep = ((ids >= 0) & (ids < s["vocab"]) & (acts < s["actions"])).nonzero()[:, 0]
    item = torch.zeros(s["vocab"], D, device="cuda", dtype=torch.float64)
    item.index_put_((ids[keep],), rows[keep], accumulate=True)
    action = torch.stack([rows[keep][acts[keep] == a].sum(0) for a in range(s["actions"])])
    return {"d_item": item, "d_action": action}


def exact_adamw(s):
    step = s["step"] + 1
    out = {name: [] for name in updated(s)}
    for b, end, w in zip(s["starts"], s["ends"].tolist(), s["decay"].tolist()):
        for a in range(b, end, 1 << 25):
            e = min(a + (1 << 25), end)
            state = {"m": s["m"][a:e].double(), "v": s["v"][a:e].double()}
            if s["bits"] == 8:
                for name in state:
                    state[name] = state[name] * s[name + "_scale"][a // BLOCK:e // BLOCK].double().repeat_interleave(BLOCK)
                state["v"] = state["v"] ** 2
            g = s["grad"][a:e].double()
            m = BETA1 * state["m"] + (1 - BETA1) * g
            v = BETA2 * state["v"] + (1 - BETA2) * g ** 2
            hat_m, hat_v = m / (1 - BETA1 ** step), v / (1 - BETA2 ** step)
            p = s["param"][a:e].double()
            p = p - LR * (w * p + hat_m / (hat_v.sqrt() + EPS))
            got = {"param": p, "m": m, "v": v, "copy": p}
            if s["bits"] == 8:
                for name, x in (("m", m), ("v", v.sqrt())):
                    top = x.view(-1, BLOCK).abs().amax(1)
                    got[name + "_scale"] = torch.where(top >= SCALE_MIN, top / E4M3_MAX, 0.0)
                    y = x / got[name + "_scale"].clamp_min(2.0 ** -120).repeat_interleave(BLOCK)
                    if name == "v":
                        y = torch.where(y > 0, y.clamp_min(E4M3_TINY), y)
                    got[name] = y.to(torch.float8_e4m3fn).double()
            for name in out:
                out[name].append(got[name])
    return {name: torch.cat(parts) for name, parts in out.items()}
