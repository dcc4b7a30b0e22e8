"""Cases, plain forms and calls for measuring the 4-bit group-scale linear
(bitlinear.forward_w4) and the sampler (bitlinear.sample).

With `own` false, `run` computes the operators with elementary torch
operations; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2}


def listed():
    return [
        # One token through a square projection of the decode layer set: the call's latency counts.
        {"name": "w4_o_m1", "op": "w4", "M": 1, "K": 2560, "N": 2560, "group": 128, "x": "fp32", "scale": "fp32"},
        # One token through the widest projection, the finest groups.
        {"name": "w4_gate_up_m1", "op": "w4", "M": 1, "K": 2560, "N": 13824, "group": 32, "x": "bf16",
         "scale": "bf16"},
        # One token through an output head: the largest weight stream of a decode step.
        {"name": "w4_head_m1", "op": "w4", "M": 1, "K": 2560, "N": 128000, "group": 128, "x": "bf16",
         "scale": "bf16"},
        # A batch of sixteen sequences through a head of an odd vocabulary, fp32 activations.
        {"name": "w4_head_m16", "op": "w4", "M": 16, "K": 1024, "N": 50021, "group": 64, "x": "fp32",
         "scale": "fp32"},
        # Vision-sized layer, a ragged number of tokens.
        {"name": "w4_vision_m250", "op": "w4", "M": 250, "K": 1152, "N": 4304, "group": 32, "x": "bf16",
         "scale": "bf16"},
        # Prompt of 512 tokens, long rows, fp32 activations.
        {"name": "w4_down_m512", "op": "w4", "M": 512, "K": 6912, "N": 2560, "group": 128, "x": "fp32",
         "scale": "fp32"},
        # Prompt of 4096 tokens through the widest projection: the largest call.
        {"name": "w4_gate_up_m4096", "op": "w4", "M": 4096, "K": 2560, "N": 13824, "group": 128, "x": "bf16",
         "scale": "bf16"},
        # One sequence, the usual chat settings.
        {"name": "sample_b1", "op": "sample", "B": 1, "V": 128000, "logits": "fp32", "mode": "chat"},
        # Small vocabulary, every token may be drawn.
        {"name": "sample_b32_plain", "op": "sample", "B": 32, "V": 32000, "logits": "fp32", "mode": "plain"},
        # A serving batch in which every sequence brings its own settings; bf16 logits hold many ties.
        {"name": "sample_b64_mixed", "op": "sample", "B": 64, "V": 50021, "logits": "bf16", "mode": "mixed"},
        # A large batch with a nucleus only: thousands of tokens stay in.
        {"name": "sample_b256_nucleus", "op": "sample", "B": 256, "V": 128000, "logits": "fp32", "mode": "nucleus"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        while True:
            M = _log_int(rng, 1, 4096)
            K = 16 * _log_int(rng, 16, 512)
            N = _log_int(rng, 64, 128000)
            if M * N * K <= 4096 * 13824 * 2560 and N * K <= 128000 * 2560 and M * N <= 4096 * 13824:
                break
        return {"op": "w4", "M": M, "K": K, "N": N, "group": rng.choice([32, 64, 128]),
                "x": rng.choice(["fp32", "bf16"]), "scale": rng.choice(["fp32", "bf16"])}
    return {"op": "sample", "B": _log_int(rng, 1, 256), "V": _log_int(rng, 1000, 128000),
            "logits": rng.choice(["fp32", "bf16"]), "mode": rng.choice(["chat", "plain", "mixed", "nucleus"])}


# ------------------------------------------------------------------- inputs

def _w4_inputs(case, seed):
    """x, 4-bit codes two to a byte (low nibble first, stored + 8) and group
    scales, as a checkpoint holds them."""
    M, K, N, g = case["M"], case["K"], case["N"], case["group"]
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    x = torch.randn((M, K), generator=gen, device="cuda")
    outlier = torch.rand((K,), generator=gen, device="cuda") < 0.01  # heavy channels
    x = torch.where(outlier, x * 20.0, x).to(DTYPES[case["x"]])
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for n in range(0, N, step):  # codes of normally distributed weights, absmax at 7
        c = (torch.randn((min(step, N - n), K), generator=gen, device="cuda") * 2.6).round_().clamp_(-8, 7).add_(8)
        c = c.to(torch.uint8)
        codes[n:n + step] = c[:, 0::2] | (c[:, 1::2] << 4)
    S = (0.02 / 2.6) * (0.6 + 0.8 * torch.rand((N, -(-K // g)), generator=gen, device="cuda"))
    return x, codes, S.to(DTYPES[case["scale"]])


def _sample_inputs(case, seed):
    """Logits of a language model's shape (a broad body, a few likely tokens,
    some rows with forbidden tokens), uniform numbers and the rows' settings."""
    B, V, mode = case["B"], case["V"], case["mode"]
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    x = torch.randn((B, V), generator=gen, device="cuda") * (1.5 + 1.5 * rand(B, 1))
    hot = torch.randint(0, V, (B, 24), generator=gen, device="cuda")
    x.scatter_(1, hot, 6.0 + 6.0 * rand(B, 24))
    kind = torch.arange(B, device="cuda").add_(seed).remainder_(8)
    banned = rand(B, V) < 0.9
    x = torch.where(banned & (kind == 3)[:, None], torch.full_like(x, -math.inf), x)
    x = torch.where(banned & (kind == 5)[:, None], torch.full_like(x, torch.finfo(DTYPES[case["logits"]]).min), x)
    x = x.to(DTYPES[case["logits"]])
    u = rand(B)
    T = 0.5 + rand(B)
    k = torch.zeros(B, dtype=torch.int32, device="cuda")
    p = torch.ones(B, device="cuda")
    m = torch.zeros(B, device="cuda")
    if mode == "chat":
        k, p = k + 50, p * 0.95
    elif mode == "nucleus":
        p = 0.8 + 0.19 * rand(B)
    elif mode == "mixed":
        kk = torch.exp(rand(B) * math.log(1000.0)).to(torch.int32)
        k = torch.where(rand(B) < 0.5, kk, k)
        p = torch.where(rand(B) < 0.5, 0.5 + 0.5 * rand(B), p)
        m = torch.where(rand(B) < 0.3, 0.1 * rand(B), m)
        T = torch.where(rand(B) < 0.1, torch.zeros_like(T), T)
    return x, u, T, k, p, m


def prepare(case, seed):
    if case["op"] == "w4":
        x, codes, S = _w4_inputs(case, seed)
        if own:
            from bit_ternary_b200 import bitlinear as BL
            packed = BL.import_w4(codes, S, case["group"])  # laid out once, as for a loaded checkpoint
            ws = torch.zeros(BL.w4_workspace_size(case["M"], case["N"], case["K"]), dtype=torch.uint8, device="cuda")
            return {"case": case, "x": x, "packed": packed, "ws": ws}
        return {"case": case, "x": x, "codes": codes, "S": S}
    x, u, T, k, p, m = _sample_inputs(case, seed)
    return {"case": case, "logits": x, "u": u, "temperature": T, "top_k": k, "top_p": p, "min_p": m}


# --------------------------------------------------------------- plain forms

def _w4_plain(x, codes, S, group):
    N, K = codes.shape[0], codes.shape[1] * 2
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(N, K).to(torch.float32) - 8.0
    W = c * S.float().repeat_interleave(group, dim=1)[:, :K]
    return x.float() @ W.t()


def _sample_plain(x, u, T, k, p, m):
    B, V = x.shape
    z = x.double()
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    valid = z > -math.inf
    order = torch.sort(z, dim=1, descending=True, stable=True).indices  # equal values keep index order
    z = torch.gather(z, 1, order)
    top = z[:, :1]
    Td = T.double()[:, None]
    greedy = ~(Td > 0)
    w = torch.exp((z - top) / torch.where(greedy, torch.ones_like(Td), Td))
    w = torch.where(z == top, torch.ones_like(w), w)
    w = torch.where(torch.gather(valid, 1, order), w, torch.zeros_like(w))
    rank = torch.arange(V, device=x.device)
    limit = torch.where(k > 0, k, torch.full_like(k, V))[:, None]
    w = torch.where(rank < limit, w, torch.zeros_like(w))
    run = torch.cumsum(w, 1)
    pd = p.double()[:, None]
    inside = (run - w < pd * run[:, -1:]) | (pd >= 1) | (rank == 0)
    w = torch.where(inside, w, torch.zeros_like(w))
    w = torch.where(w >= m.double().clamp(max=1.0)[:, None], w, torch.zeros_like(w))
    w = torch.where(greedy & (rank > 0), torch.zeros_like(w), w)
    w = torch.zeros_like(w).scatter_(1, order, w)  # back to index order
    run = torch.cumsum(w, 1)
    total = run[:, -1]
    hit = run > (u.double() * total)[:, None]
    token = hit.to(torch.uint8).argmax(1)
    prob = torch.gather(w, 1, token[:, None])[:, 0]
    logprob = torch.log(prob / total).float()
    none = ~valid.any(1)
    return (torch.where(none, torch.full_like(token, -1), token),
            torch.where(none, torch.full_like(logprob, -math.inf), logprob))


def run(state):
    case = state["case"]
    if case["op"] == "w4":
        if own:
            from bit_ternary_b200 import bitlinear as BL
            return BL.forward_w4(state["x"], state["packed"], ws=state["ws"])
        return _w4_plain(state["x"], state["codes"], state["S"], case["group"])
    args = (state["logits"], state["u"], state["temperature"], state["top_k"], state["top_p"], state["min_p"])
    if own:
        from bit_ternary_b200 import bitlinear as BL
        return BL.sample(*args)
    return _sample_plain(*args)


def work(case):
    if case["op"] == "w4":
        M, K, N = case["M"], case["K"], case["N"]
        scales = N * -(-K // case["group"]) * BYTES[case["scale"]]
        return {"bytes": N * K // 2 + scales + M * K * BYTES[case["x"]] + 4 * M * N, "flops": 2 * M * N * K}
    B, V = case["B"], case["V"]
    # per token: a comparison, a difference, a product, an exponential, a sum
    return {"bytes": B * V * BYTES[case["logits"]] + B * (4 + 16 + 8 + 4), "flops": 5 * B * V}


# ---------------------------------------------------------- 64-bit definition

def _w4_exact(case, seed):
    x, codes, S = _w4_inputs(case, seed)
    M, K, N, g = case["M"], case["K"], case["N"], case["group"]
    xd = x.double()
    y = torch.empty((M, N), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // K)
    for n in range(0, N, step):
        b = codes[n:n + step]
        c = torch.empty((b.shape[0], K), dtype=torch.float64, device="cuda")
        c[:, 0::2] = b.remainder(16)
        c[:, 1::2] = torch.div(b, 16, rounding_mode="floor")
        c -= 8
        for G in range(S.shape[1]):
            c[:, G * g:(G + 1) * g] *= S[n:n + step, G:G + 1].double()
        y[:, n:n + step] = xd @ c.t()
    return y


def _sample_exact(case, seed):
    x, u, T, k, p, m = [t.double().cpu().numpy() for t in _sample_inputs(case, seed)]
    tokens, logprobs = [], []
    for r in range(case["B"]):
        row = x[r]
        idx = np.flatnonzero(~np.isnan(row) & (row != -np.inf))
        if idx.size == 0:
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        best = row[idx].max()
        if not T[r] > 0:
            tokens.append(int(idx[row[idx] == best][0]))
            logprobs.append(0.0)
            continue
        idx = idx[np.argsort(-row[idx], kind="stable")]  # value descending, index ascending
        if k[r] > 0:
            idx = idx[:int(k[r])]
        w = np.exp((row[idx] - best) / T[r])
        if p[r] < 1:
            run = np.cumsum(w)
            n = 1 + int(np.searchsorted(run, p[r] * run[-1], side="left"))
            idx, w = idx[:n], w[:n]
        keep = w >= min(m[r], 1.0)
        idx, w = idx[keep], w[keep]
        back = np.argsort(idx)
        idx, w = idx[back], w[back]
        run = np.cumsum(w)
        j = min(int(np.searchsorted(run, u[r] * run[-1], side="right")), idx.size - 1)
        tokens.append(int(idx[j]))
        logprobs.append(math.log(w[j] / run[-1]))
    return (torch.tensor(tokens, dtype=torch.int64, device="cuda"),
            torch.tensor(logprobs, dtype=torch.float64, device="cuda"))


def exact(case, seed):
    return _w4_exact(case, seed) if case["op"] == "w4" else _sample_exact(case, seed)
