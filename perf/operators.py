"""Linear layers over Leech-lattice compressed weights: cases, inputs and plain forms.

    linear   y = act(x W^T + b) + r           for every token of a batch
    grouped  the same with one weight per expert, the tokens sorted by expert

With `gated` the weight rows are [gate; up] and y = act(gate) * up + r.  W is held as packed 48-bit
block indices with a gain code (24 weights per word); the plain forms below decode it with ordinary
tensor operations.  The index format: shells m = 2..13 of the Leech lattice in order, in a shell the
even coset's classes before the odd coset's, classes by their magnitudes (descending, compared
lexicographically); in a class I = r + A (s + 2^B p) with the codeword r, the signs s and the
arrangement rank p.
"""
import functools
import itertools
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
MAX_SHELL = 13
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---- the index format ---------------------------------------------------------------------------
def _codewords():
    """The 4096 words of the extended Golay code, ascending."""
    g = sum(1 << e for e in (0, 2, 4, 5, 6, 10, 11))
    words = [0]
    for i in range(12):
        row = g << i
        row |= (bin(row).count("1") & 1) << 23
        words += [w ^ row for w in words]
    return sorted(words)


def _multisets(values, places, squares):
    """Multisets (descending tuples of (value, count)) of `places` values with that sum of squares."""
    if not values:
        return [()] if places == 0 and squares == 0 else []
    v, rest, found = values[0], values[1:], []
    for c in range(places + 1):
        if c * v * v > squares:
            break
        found += [(((v, c),) if c else ()) + t for t in _multisets(rest, places - c, squares - c * v * v)]
    return found


def _arrangements(counts):
    n = math.factorial(sum(counts))
    for c in counts:
        n //= math.factorial(c)
    return n


@functools.lru_cache(None)
def _classes():
    """Every class in index order: (shell, odd, ascending ((value, count), ...), weight k, A, B, P_S, P_C, start)."""
    weights = [bin(w).count("1") for w in _codewords()]
    found, start = [], 0
    for m in range(2, MAX_SHELL + 1):
        for odd in (0, 1):
            top = math.isqrt(16 * m)
            values = [v for v in range(top, -1, -1) if v % 2 == odd]
            group = []
            for t in _multisets(values, 24, 16 * m):
                if odd:
                    ok = sum((v if v % 4 == 3 else -v) * c for v, c in t) % 8 == 4
                    k, a, b = 0, 4096, 0
                    ps, pc = 1, _arrangements([c for _, c in t])
                else:
                    k = sum(c for v, c in t if v % 4 == 2)
                    a = weights.count(k)
                    ok = a > 0 and (k > 0 or sum(v * c for v, c in t) % 8 == 0)
                    b = sum(c for v, c in t if v) - (k > 0)
                    ps = _arrangements([c for v, c in t if v % 4 == 2])
                    pc = _arrangements([c for v, c in t if v % 4 == 0])
                if ok:
                    order = tuple(itertools.chain.from_iterable((v,) * c for v, c in t))
                    group.append((order, (m, odd, t[::-1], k, a, b, ps, pc)))
            for _, c in sorted(group):
                found.append(c + (start,))
                start += c[4] * c[6] * c[7] << c[5]
    return found, start


@functools.lru_cache(None)
def _tables():
    """The classes' constants as tensors, for the plain form."""
    classes, _ = _classes()
    most = max(len(c[2]) for c in classes)
    words = _codewords()
    by_weight = sorted(words, key=lambda w: (bin(w).count("1"), w))
    base = {k: next(i for i, w in enumerate(by_weight) if bin(w).count("1") == k) for k in (0, 8, 12, 16, 24)}
    pad = [c[2] + ((0, 0),) * (most - len(c[2])) for c in classes]
    long = functools.partial(torch.tensor, dtype=torch.int64, device=DEVICE)
    return {
        "start": long([c[8] for c in classes]), "A": long([c[4] for c in classes]), "B": long([c[5] for c in classes]),
        "PS": long([c[6] for c in classes]), "PC": long([c[7] for c in classes]),
        "odd": long([c[1] for c in classes]), "shell": long([c[0] for c in classes]), "k": long([c[3] for c in classes]),
        "word0": long([4096 if c[1] else base[c[3]] for c in classes]),
        "words": long(by_weight + words),
        "parity": long([sum(v * n for v, n in c[2]) // 4 % 2 for c in classes]),
        # one row per magnitude group, one column per class
        "value": long([[p[i][0] for p in pad] for i in range(most)]),
        "count": long([[p[i][1] for p in pad] for i in range(most)]),
        "inside": long([[int(not c[1] and p[i][0] % 4 == 2) for c, p in zip(classes, pad)] for i in range(most)]),
    }


def _points(index):
    """Lattice points [n, 24] (int64) and shells [n] of block indices, all blocks side by side."""
    t = _tables()
    c = torch.searchsorted(t["start"], index, right=True) - 1
    i = index - t["start"][c]
    r, i = i % t["A"][c], i // t["A"][c]
    s, p = i & ((1 << t["B"][c]) - 1), i >> t["B"][c]
    word = t["words"][t["word0"][c] + r]
    odd = t["odd"][c].bool()
    inside_groups, value, count = t["inside"][:, c].bool(), t["value"][:, c], t["count"][:, c]
    on = torch.where(odd, 0, word)                                   # positions of the second coordinate set
    ranks = [torch.where(odd, p, p // t["PS"][c]), torch.where(odd, 0, p % t["PS"][c])]
    ways = [t["PC"][c], t["PS"][c]]
    left = [24 - t["k"][c], t["k"][c]]
    size = []
    for q in range(24):
        here = (on >> q & 1).bool()
        rank, way, places = (torch.where(here, b, a) for a, b in (ranks, ways, left))
        mine = count * (inside_groups == here)
        upto = mine.cumsum(0)
        pick = (rank * places >= way * upto).sum(0, keepdim=True)
        n = mine.gather(0, pick)[0]
        rank = rank - way * (upto.gather(0, pick)[0] - n) // places
        way = way * n // places
        size.append(value.gather(0, pick)[0])
        count.scatter_add_(0, pick, torch.full_like(pick, -1))
        ranks = [torch.where(here, ranks[0], rank), torch.where(here, rank, ranks[1])]
        ways = [torch.where(here, ways[0], way), torch.where(here, way, ways[1])]
        left = [torch.where(here, left[0], places - 1), torch.where(here, places - 1, left[1])]
    size = torch.stack(size, 1)
    bit = word[:, None] >> torch.arange(24, device=word.device) & 1
    sign_odd = torch.where((bit == 1) == (size % 4 == 1), 1, -1)
    # even coset: one sign bit per nonzero coordinate, but for the highest of the codeword
    top = (bit * torch.arange(1, 25, device=word.device)).amax(1, keepdim=True) - 1
    free = (size != 0) & (torch.arange(24, device=word.device) != top)
    place = free.cumsum(1) - 1
    negative = free & (s[:, None] >> place.clamp(min=0) & 1).bool()
    wrong = ((negative & (bit == 1)).sum(1, keepdim=True) + t["parity"][c][:, None]) % 2 == 1
    negative = negative | (wrong & (torch.arange(24, device=word.device) == top))
    sign = torch.where(odd[:, None], sign_odd, torch.where(negative, -1, 1))
    return size * sign, t["shell"][c]


# ---- the cases ----------------------------------------------------------------------------------
def _case(name, op, tokens, rows, cols, dtype="float16", activation="none", gated=False, bias=False, residual=False,
          gain="table", experts=1, spare=0):
    """rows: outputs of the layer (a gated weight has twice as many); tokens: rows of x in use; spare:
    rows of x and y behind them."""
    c = dict(op=op, tokens=tokens, rows=rows, cols=cols, dtype=dtype, activation=activation, gated=gated, bias=bias,
             residual=residual, gain=gain, experts=experts, spare=spare)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one sequence through an attention output projection, added to the stream
        _case("one token", "linear", 1, 4096, 4096, residual=True),
        # one token through the gate and up projections of an MLP, the widest layer of a 7B decoder
        _case("one token gated", "linear", 1, 11008, 4096, "bfloat16", "silu", True),
        # eight sequences decoding together, the MLP's way down
        _case("eight tokens down", "linear", 8, 4096, 11008, residual=True),
        # a larger serving batch, a layer with a bias and the tanh form of gelu
        _case("sixty-four tokens", "linear", 64, 4096, 4096, "bfloat16", "gelu_tanh", bias=True),
        # odd everything: a classifier head or an adapter's projection, a gain per block
        _case("odd sizes", "linear", 333, 1001, 999, "float16", "gelu", bias=True, residual=True, gain="direct"),
        # a prompt of a thousand tokens through the gated MLP
        _case("prompt gated", "linear", 1024, 11008, 4096, "bfloat16", "silu", True),
        # prefill of four thousand tokens, the way down
        _case("prefill down", "linear", 4096, 4096, 11008, residual=True),
        # a 70B decoder's widest layer on a prompt
        _case("wide layer", "linear", 2048, 28672, 8192, "bfloat16", "relu", bias=True),
        # two sequences, eight experts each of sixty-four: most experts have no token
        _case("few tokens, many experts", "grouped", 16, 1408, 2048, "bfloat16", "silu", True, experts=64),
        # odd sizes, a padded batch
        _case("odd experts", "grouped", 77, 331, 1000, "float16", "gelu", bias=True, residual=True, experts=5, spare=19),
        # a serving batch over eight wide experts
        _case("eight experts", "grouped", 512, 5504, 4096, "float16", "silu", True, experts=8),
        # a long prompt over sixteen experts, the way down
        _case("prompt over experts", "grouped", 8192, 2048, 5504, "bfloat16", experts=16, spare=128),
    ]


LARGEST = 2 * 2048 * 28672 * 8192                     # flops of the largest listed case
WEIGHTS = 28672 * 8192                                # weights of the largest layer


def _spread(rng, low, high):
    """A whole number spread evenly over the logarithm of [low, high]; one in three a multiple of 64."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(64, n // 64 * 64) if high >= 64 and n >= 64 and rng.random() < 1 / 3 else n


def draw(rng):
    op = rng.choice(("linear", "grouped"))
    while True:
        experts = _spread(rng, 2, 96) if op == "grouped" else 1
        rows, cols, gated = _spread(rng, 24, 28672), _spread(rng, 24, 28672), rng.random() < 0.4
        tokens = _spread(rng, 1, 8192)
        weights = experts * rows * cols * (2 if gated else 1)
        if weights <= WEIGHTS and 2 * tokens * rows * cols * (2 if gated else 1) <= LARGEST:
            break
    return _case(None, op, tokens, rows, cols, rng.choice(("float16", "bfloat16")), rng.choice(ACTIVATIONS), gated,
                 rng.random() < 0.4, rng.random() < 0.4, rng.choice(("table", "table", "direct")), experts,
                 rng.choice((0, rng.randint(1, 64))) if op == "grouped" else 0)


# ---- inputs -------------------------------------------------------------------------------------
def prepare(case, seed):
    """A compressed layer and its activations.  Blocks are uniform over the coded points (what a
    Gaussian source's nearest points look like to a decoder); gains follow the norm of 24 Gaussian
    weights with a spread of scales over the rows; a few channels of x are far larger than the rest."""
    g = torch.Generator(DEVICE).manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    cols, experts = case["cols"], case["experts"]
    rows = case["rows"] * (2 if case["gated"] else 1)
    blocks = -(-cols // 24)
    tokens = case["tokens"] + case["spare"]
    f32 = dict(dtype=torch.float32, device=DEVICE, generator=g)
    index = torch.randint(0, _classes()[1], (experts * rows, blocks), dtype=torch.int64, device=DEVICE, generator=g)
    scale = (torch.rand(experts * rows, 1, **f32) * 1.5 + 0.5) / math.sqrt(cols)
    if case["gain"] == "table":
        # quantiles of the norm of 24 Gaussian values (cube-root approximation), one table per row
        u = torch.special.ndtri((torch.arange(256, dtype=torch.float64, device=DEVICE) + 0.5) / 256)
        norm = (24 * (1 - 2 / 216 + u * math.sqrt(2 / 216)) ** 3).sqrt().float()
        gains = (scale * norm).half()
        code = torch.randint(0, 256, index.shape, dtype=torch.int64, device=DEVICE, generator=g)
        words = index | code << 48
    else:
        # a scale per block: the block's norm over |v|, about 4 sqrt(12.8)
        gains = (scale * torch.randn(index.shape, **f32).mul_(0.14).add_(1) * (math.sqrt(24) / 14.3)).half()
        words = index
    x = torch.randn(tokens, cols, **f32)
    x[:, torch.randint(0, cols, (1 + cols // 512,), device=DEVICE, generator=g)] *= 12
    state = dict(case=dict(case), words=words, gains=gains, x=x.to(dtype), bias=None, residual=None)
    if case["bias"]:
        state["bias"] = (torch.randn(experts * rows, **f32) * 0.5).to(dtype)
    if case["residual"]:
        state["residual"] = torch.randn(tokens, case["rows"], **f32).to(dtype)
    state["y"] = torch.randn(tokens, case["rows"], **f32).to(dtype)       # rows in spare keep these
    if case["op"] == "grouped":
        # uneven shares, some experts without a token
        share = torch.randn(experts, **f32).mul_(1.2).exp_() * (torch.rand(experts, **f32) > 0.15)
        share[0] += 1e-3
        chosen = torch.multinomial(share, case["tokens"], replacement=True, generator=g)
        counts = torch.bincount(chosen, minlength=experts)
        state["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).int()
        state["most"] = int(counts.max())
    return state


# ---- one pass -----------------------------------------------------------------------------------
@functools.lru_cache(None)
def _codec():
    import codebook_free_lattice_b200 as llvq
    return llvq, llvq.Codec(48)


def _run_own(state):
    llvq, codec = _codec()
    case = state["case"]
    if "weight" not in state:
        mode = llvq.LLVQ_GAIN_U8_TABLE if case["gain"] == "table" else llvq.LLVQ_GAIN_FP16_DIRECT
        state["weight"] = codec.weight(state["words"], state["gains"], state["words"].shape[0], case["cols"], mode)
        state["activation"] = getattr(llvq, "LLVQ_ACT_" + case["activation"].upper())
        state["workspace"] = None
    ends = dict(bias=state["bias"], activation=state["activation"], gated=case["gated"], residual=state["residual"],
                workspace=state["workspace"])
    if case["op"] == "linear":
        state["workspace"] = codec.linear(state["weight"], state["x"], state["y"], **ends)
    else:
        state["workspace"] = codec.linear_grouped(state["weight"], case["experts"], state["x"], state["offsets"],
                                                  state["y"], **ends)
    return state["y"]


def _activate(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _weights(state):
    """The dense weight [experts * rows, cols] in 32 bits."""
    case, words = state["case"], state["words"]
    points, shell = _points((words & (1 << 48) - 1).reshape(-1))
    if case["gain"] == "table":
        gain = state["gains"].float().gather(1, words >> 48).reshape(-1) / (4 * shell.float().sqrt())
    else:
        gain = state["gains"].float().reshape(-1)
    return (points.float() * gain[:, None]).reshape(words.shape[0], -1)[:, :case["cols"]]


def _epilogue(z, state, bias, residual):
    if bias is not None:
        z = z + bias.float()
    if state["case"]["gated"]:
        gate, up = z.chunk(2, -1)
        z = _activate(gate, state["case"]["activation"]) * up
    else:
        z = _activate(z, state["case"]["activation"])
    return z if residual is None else z + residual.float()


def run(state):
    if own:
        return _run_own(state)
    case, x = state["case"], state["x"].float()
    weight = _weights(state)
    if case["op"] == "linear":
        return _epilogue(x @ weight.t(), state, state["bias"], state["residual"]).to(state["x"].dtype)
    # every expert's tokens side by side, padded to the longest
    experts, offsets = case["experts"], state["offsets"].long()
    at = offsets[:-1, None] + torch.arange(state["most"], device=x.device)
    used = at < offsets[1:, None]
    z = x[at.clamp(max=x.shape[0] - 1)] @ weight.reshape(experts, -1, case["cols"]).transpose(1, 2)
    bias = None if state["bias"] is None else state["bias"].reshape(experts, 1, -1)
    residual = None if state["residual"] is None else state["residual"][at.clamp(max=x.shape[0] - 1)]
    y = _epilogue(z, state, bias, residual).to(state["x"].dtype)
    # padding goes to a row of its own, which is then cut off
    out = torch.cat((state["y"], state["y"][:1]))
    out[torch.where(used, at, x.shape[0]).reshape(-1)] = y.reshape(-1, case["rows"])
    return out[:-1]


def work(case):
    rows = case["rows"] * (2 if case["gated"] else 1)
    blocks, tokens = -(-case["cols"] // 24), case["tokens"]
    used = min(case["experts"], tokens)                   # experts that can have a token
    weight = used * rows * (8 * blocks + (512 if case["gain"] == "table" else 2 * blocks))
    rest = 2 * tokens * (case["cols"] + case["rows"] * (2 if case["residual"] else 1))
    return {"bytes": weight + rest + (2 * used * rows if case["bias"] else 0), "flops": 2 * tokens * rows * case["cols"]}


# ---- the definition in 64 bits ------------------------------------------------------------------
def _unrank(rank, groups):
    """Arrangements [n, length] of a multiset ((value, count), ascending) by lexicographic rank: at each
    place, the arrangements that begin with a smaller value are counted off one value after the other."""
    n, length = rank.shape[0], sum(c for _, c in groups)
    out = rank.new_zeros(n, length)
    left = [torch.full_like(rank, c) for _, c in groups]
    total = torch.full_like(rank, _arrangements([c for _, c in groups]))
    rank = rank.clone()
    for q in range(length):
        done = torch.zeros_like(rank, dtype=torch.bool)
        following = torch.zeros_like(rank)
        for (value, _), c in zip(groups, left):
            starting = total * c // (length - q)
            chosen = ~done & (rank < starting)
            out[:, q] += value * chosen
            following += starting * chosen
            rank -= starting * (~done & ~chosen)
            c -= chosen.long()
            done |= chosen
        total = following
    return out


def _define_weight(words, gains, table):
    """The dense weight in 64 bits, one class of blocks after another."""
    classes, _ = _classes()
    index = (words & (1 << 48) - 1).reshape(-1)
    vectors = torch.zeros(index.numel(), 24, dtype=torch.float64, device=words.device)
    norms = torch.ones(index.numel(), dtype=torch.float64, device=words.device)
    code = _codewords()
    order = index.argsort()
    edges = torch.searchsorted(index[order], torch.tensor([c[8] for c in classes], device=words.device)).tolist() + [index.numel()]
    for j, (m, odd, groups, k, a, b, ps, pc, start) in enumerate(classes):
        which = order[edges[j]:edges[j + 1]]
        if not which.numel():
            continue
        i = index[which] - start
        r, s, p = i % a, i // a % (1 << b), i // a >> b
        some = torch.tensor([w for w in code if odd or bin(w).count("1") == k], device=words.device)
        bits = torch.stack([some[r] >> q & 1 for q in range(24)], 1)
        if odd:
            size = _unrank(p, groups)
            # x = 1 mod 4 on the codeword, 3 mod 4 off it
            x = torch.where((size - torch.where(bits == 1, 1, 3)) % 4 == 0, size, -size)
        else:
            seats = bits.argsort(dim=1, descending=True, stable=True)   # the codeword's places, then the others
            first = _unrank(p % ps, [v for v in groups if v[0] % 4 == 2])
            second = _unrank(p // ps, [v for v in groups if v[0] % 4 == 0])
            size = torch.zeros_like(bits).scatter_(1, seats, torch.cat((first, second), 1))
            x, negatives = size.clone(), torch.zeros_like(s)
            last = torch.where(bits == 1, torch.arange(24, device=words.device), -1).amax(1)
            bit = s.clone()
            for q in range(24):
                takes = (size[:, q] != 0) & (last != q)
                minus = takes & (bit & 1 == 1)
                x[:, q] = torch.where(minus, -x[:, q], x[:, q])
                negatives += minus & (bits[:, q] == 1)
                bit = torch.where(takes, bit >> 1, bit)
            if k:
                turn = (negatives + size.sum(1) // 4) % 2 == 1
                picked = x.gather(1, last[:, None])
                x.scatter_(1, last[:, None], torch.where(turn[:, None], -picked, picked))
        vectors[which] = x.double()
        norms[which] = 4 * math.sqrt(m)
    gain = gains.double().gather(1, words >> 48).reshape(-1) / norms if table else gains.double().reshape(-1)
    return vectors.mul_(gain[:, None]).reshape(words.shape[0], -1)


def exact(case, seed):
    state = prepare(case, seed)
    dense = _define_weight(state["words"], state["gains"], case["gain"] == "table")[:, :case["cols"]]
    x, y = state["x"].double(), state["y"].double()
    if case["op"] == "linear":
        spans = [(0, 0, x.shape[0])]
    else:
        ends = np.asarray(state["offsets"].cpu()).tolist()
        spans = [(e, ends[e], ends[e + 1]) for e in range(case["experts"])]
    rows = dense.shape[0] // case["experts"]
    for e, lo, hi in spans:
        if lo == hi:
            continue
        z = torch.einsum("tk,rk->tr", x[lo:hi], dense[e * rows:(e + 1) * rows])
        if state["bias"] is not None:
            z = z + state["bias"].double()[e * rows:(e + 1) * rows]
        h = z[:, :case["rows"]]
        name = case["activation"]
        if name == "relu":
            h = torch.where(h > 0, h, 0.0)
        elif name == "silu":
            h = h * torch.sigmoid(h)
        elif name == "gelu":
            h = h * torch.special.ndtr(h)
        elif name == "gelu_tanh":
            h = h * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3))
        if case["gated"]:
            h = h * z[:, case["rows"]:]
        if state["residual"] is not None:
            h = h + state["residual"][lo:hi].double()
        y[lo:hi] = h
    return y
