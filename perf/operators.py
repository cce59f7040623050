"""Measured cases of the per-request operators of a decode batch.

lora_add       out[m] = y[m] + s[a] * (x[m] A[a]^T) B[a]^T with a = index[m]:
               low-rank adapters of many requests on the output y of a shared
               projection; a token whose index is no adapter keeps its y.
sample_logits  one token per row of logits by inverse CDF from a given random
               number, after temperature, top-p, top-k and min-p of that row.

Sizes: hidden 5120, MLP 17408, vocabulary 248320, verify chunks of 1 + 3 or
1 + 4 tokens a stream, prefill chunks of 8192 tokens (the bench's workloads);
the others are generic.
"""
import math

import numpy as np
import torch

own = False

HIDDEN, MLP, VOCAB = 5120, 17408, 248320


def _lora(name, M, K, N, R, L, run, bare):
    """run: tokens a request has in the batch; bare: share of the requests
    without an adapter."""
    return {"op": "lora_add", "name": name, "M": M, "K": K, "N": N, "R": R, "L": L, "run": run,
            "bare": bare}


def _sample(name, M, V, dtype, mode):
    """mode: "mixed" = every row its own temperature, top-k, top-p and min-p,
    a few rows greedy; "top_p" = temperature and top-p only; "plain" =
    temperature only; "masked" = as mixed, with entries masked to -inf."""
    return {"op": "sample_logits", "name": name, "M": M, "V": V, "dtype": dtype, "mode": mode}


def listed():
    return [
        # single-stream decode, one token of one adapter
        _lora("lora m1 5120-5120 r16", 1, HIDDEN, HIDDEN, 16, 4, 1, 0.0),
        # the verify chunk of one stream on the MLP's wide projection
        _lora("lora m5 5120-17408 r32", 5, HIDDEN, MLP, 32, 4, 5, 0.0),
        # decode batch of 37 requests, each with its own adapter
        _lora("lora m37 17408-5120 r64", 37, MLP, HIDDEN, 64, 48, 1, 0.1),
        # 32 streams verifying 4 tokens each
        _lora("lora m128 5120-17408 r16", 128, HIDDEN, MLP, 16, 32, 4, 0.1),
        # a chunked-prefill batch with ragged requests, sizes off every tile
        _lora("lora m1001 2056-5000 r24", 1001, 2056, 5000, 24, 6, 143, 0.2),
        # a prefill chunk of a few requests
        _lora("lora m8192 5120-17408 r16", 8192, HIDDEN, MLP, 16, 8, 1024, 0.1),
        # single-stream decode: one row of the vocabulary
        _sample("sample m1 v248320", 1, VOCAB, "bfloat16", "mixed"),
        # one stream's verify chunk, fp32 logits masked by a grammar
        _sample("sample m5 v248320 f32", 5, VOCAB, "float32", "masked"),
        # a small odd vocabulary
        _sample("sample m8 v5003", 8, 5003, "bfloat16", "top_p"),
        # a decode batch, odd vocabulary, whole softmax
        _sample("sample m33 v32003 f32", 33, 32003, "float32", "plain"),
        # 32 streams verifying 4 tokens each
        _sample("sample m128 v248320", 128, VOCAB, "bfloat16", "mixed"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        K, N = (8 * _spread(rng, 64, MLP // 8) for _ in range(2))
        R = rng.choice([8, 16, 24, 32, 64, 96, 128])
        L = _spread(rng, 1, 64)
        # no more than the largest listed case's tokens and adapter bytes
        most = 8192 * (HIDDEN + MLP)
        L = max(1, min(L, most // (R * (K + N))))
        M = _spread(rng, 1, 8192)
        M = max(1, min(M, most // (K + N), 8192 * 128 // (L * R)))
        return {"op": "lora_add", "M": M, "K": K, "N": N, "R": R, "L": L,
                "run": _spread(rng, 1, 1024), "bare": rng.choice([0.0, 0.1, 0.3])}
    V = _spread(rng, 256, VOCAB)
    return {"op": "sample_logits", "M": max(1, min(_spread(rng, 1, 256), 128 * VOCAB // V)), "V": V,
            "dtype": rng.choice(["bfloat16", "float32"]),
            "mode": rng.choice(["mixed", "top_p", "plain", "masked"])}


def _prepare_lora(c, g, dev):
    M, K, N, R, L = c["M"], c["K"], c["N"], c["R"], c["L"]

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(scale)
    requests = -(-M // c["run"])
    which = torch.randint(0, L, (requests,), generator=g, device=dev)
    which[torch.rand(requests, generator=g, device=dev) < c["bare"]] = -1
    index = which.repeat_interleave(c["run"])[:M].to(torch.int32).contiguous()
    return {
        "x": randn(M, K).bfloat16(),
        "a": randn(L, R, K, scale=K ** -0.5).bfloat16(),
        "b": randn(L, N, R, scale=R ** -0.5).bfloat16(),
        "scales": torch.rand(L, generator=g, device=dev) + 0.5,
        "index": index,
        "y": randn(M, N).bfloat16(),
    }


def _choice(values, M, g, dev, dtype):
    return torch.tensor(values, device=dev, dtype=dtype)[
        torch.randint(0, len(values), (M,), generator=g, device=dev)]


def _prepare_sample(c, g, dev):
    M, V, mode = c["M"], c["V"], c["mode"]
    # a bell-shaped bulk and some raised candidates, as trained heads give
    logits = torch.randn(M, V, generator=g, device=dev).mul_(2.2)
    at = torch.randint(0, V, (M, 48), generator=g, device=dev)
    logits.scatter_add_(1, at, torch.empty(M, 48, device=dev).exponential_(0.2, generator=g))
    if mode == "masked":
        logits.masked_fill_(torch.rand(M, V, generator=g, device=dev) < 0.4, float("-inf"))
    mixed = mode in ("mixed", "masked")
    return {
        "logits": logits.to(getattr(torch, c["dtype"])),
        "u": torch.rand(M, generator=g, device=dev),
        "temperature": _choice([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.3] if mixed else [0.7, 0.8, 1.0], M,
                               g, dev, torch.float32),
        "top_k": _choice([0, 0, 20, 50, 200, 1000], M, g, dev, torch.int32) if mixed else None,
        "top_p": None if mode == "plain" else _choice([0.8, 0.9, 0.95, 0.99], M, g, dev,
                                                      torch.float32),
        "min_p": _choice([0.0, 0.0, 0.02, 0.1], M, g, dev, torch.float32) if mixed else None,
    }


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    make = _prepare_lora if case["op"] == "lora_add" else _prepare_sample
    return {"op": case["op"], **make(case, g, dev)}


def _plain_lora(s):
    """Every adapter's inner products for every token, those of other
    adapters set to zero, then one product with all adapters' B."""
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    L, R, K = a.shape
    inner = (x @ a.reshape(L * R, K).T).reshape(-1, L, R)
    mine = s["index"].long()[:, None] == torch.arange(L, device=x.device)
    inner = torch.where(mine[:, :, None], inner * s["scales"][:, None], 0.0).reshape(-1, L * R)
    delta = inner @ b.permute(0, 2, 1).reshape(L * R, -1)
    return (s["y"].float() + delta).bfloat16()


def _plain_sample(s):
    """Sort, cumulative sums and comparisons in 64 bits: a token is picked
    where a cumulative sum crosses a border."""
    z = s["logits"].double()
    M, V = z.shape
    z = torch.where(torch.isnan(z), -math.inf, z)
    top = z.max(dim=1, keepdim=True).values
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    t = torch.where(greedy, 1.0, t)
    w = torch.where(z == top, 1.0, torch.exp((z - top) / t))
    ranked, order = torch.sort(z, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        cum = ws.cumsum(1)
        before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
        keep &= (before < p * cum[:, -1:]) | (p >= 1)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (torch.arange(V, device=z.device) < k) | (k <= 0)
    if s["min_p"] is not None:
        q = s["min_p"].double()[:, None]
        floor = torch.log(q.clamp(max=1.0)) * t
        keep &= (ranked - top >= floor) | ~(q > 0)
    keep = torch.where(greedy, ranked == top, keep)
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
    cum = kept.cumsum(1)
    total = cum[:, -1:]
    over = cum > s["u"].double()[:, None] * total
    pick = torch.where(over.any(1), over.to(torch.uint8).argmax(1), V - 1)
    pick = torch.where(greedy[:, 0], order[:, 0], pick)
    prob = torch.where(greedy[:, 0], 1.0, kept.gather(1, pick[:, None])[:, 0] / total[:, 0])
    return {"tokens": pick.to(torch.int32), "probs": prob.float()}


def run(state):
    if own:
        import mxfp8_gemm_speculative_b200 as mxg
        if state["op"] == "lora_add":
            return mxg.lora_add(state["x"], state["a"], state["b"], state["index"], state["y"],
                                scales=state["scales"])
        tokens, probs = mxg.sample_logits(state["logits"], state["u"], state["temperature"],
                                          state["top_k"], state["top_p"], state["min_p"])
        return {"tokens": tokens, "probs": probs}
    return _plain_lora(state) if state["op"] == "lora_add" else _plain_sample(state)


def work(case):
    M = case["M"]
    if case["op"] == "sample_logits":
        size = 2 if case["dtype"] == "bfloat16" else 4
        # logits, random number and parameters in; token and probability out
        return {"bytes": M * case["V"] * size + M * (20 + 8), "flops": 4 * M * case["V"]}
    K, N, R, L = case["K"], case["N"], case["R"], case["L"]
    # adapters in use: distinct ones among the requests that have one
    requests = -(-M // case["run"]) * (1 - case["bare"])
    used = L * (1 - (1 - 1 / L) ** requests)
    return {"bytes": 2 * M * K + 2 * used * R * (K + N) + 4 * M * N + 4 * M + 4 * L,
            "flops": 2 * M * R * (K + N)}


def _exact_lora(s):
    x, y, index = s["x"].double(), s["y"].double(), s["index"].cpu().numpy()
    out = y.clone()
    for n in range(s["a"].shape[0]):
        rows = torch.from_numpy(np.flatnonzero(index == n)).to(x.device)
        if len(rows):
            inner = torch.einsum("mk,rk->mr", x[rows], s["a"][n].double())
            delta = torch.einsum("mr,nr->mn", inner, s["b"][n].double())
            out[rows] = y[rows] + float(s["scales"][n].double()) * delta
    return out


def _exact_sample(s):
    def host(v):
        return None if v is None else v.double().cpu().numpy()
    logits, u, temp = host(s["logits"]), host(s["u"]), host(s["temperature"])
    top_k, top_p, min_p = host(s["top_k"]), host(s["top_p"]), host(s["min_p"])
    tokens, probs = [], []
    for m, row in enumerate(logits):
        best = int(np.argmax(row))
        if not temp[m] > 0:
            tokens.append(best)
            probs.append(1.0)
            continue
        with np.errstate(invalid="ignore"):
            away = row - row[best]
            w = np.exp(away / temp[m])
        chosen = np.ones(len(row), bool)
        if top_p is not None or top_k is not None:
            rank = np.argsort(-row, kind="stable")
            if top_p is not None and top_p[m] < 1:
                sums = np.cumsum(w[rank])
                chosen[rank[1 + int(np.searchsorted(sums, top_p[m] * sums[-1], "left")):]] = False
            if top_k is not None and top_k[m] > 0:
                chosen[rank[int(top_k[m]):]] = False
        if min_p is not None and min_p[m] > 0:
            chosen &= away >= temp[m] * np.log(min_p[m])
        chosen[best] = True
        ids = np.flatnonzero(chosen & (w > 0))
        sums = np.cumsum(w[ids])
        at = min(int(np.searchsorted(sums, u[m] * sums[-1], "right")), len(ids) - 1)
        tokens.append(int(ids[at]))
        probs.append(float(w[ids[at]] / sums[-1]))
    return {"tokens": np.array(tokens, np.int32), "probs": np.array(probs, np.float64)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_lora(s) if case["op"] == "lora_add" else _exact_sample(s)
