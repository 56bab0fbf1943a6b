"""The barrier protocols of the bf16 backward kernel (both kinds of CTA) and of the tensor-core
kernel over the 8-bit cache, checked on the host.

Each role's waits, arrivals, reads and writes are restated in program order and run under many
random interleavings.  Every buffer (a shared-memory tile, a quarter of a score region in TMEM, a
slot of row terms) holds a named content, and the model checks that

* no interleaving deadlocks, and no wait for phase k of a barrier happens after phase k + 1 has
  completed (a parity wait cannot tell k from k + 2);
* a reader finds the content it wants, arrived: a TMA load lands at any later step; a product's
  result is there for threads once a commit that follows it has arrived, in issue order, and for
  later products at once;
* a content is overwritten only after all its readers are done with it: products that follow in
  issue order may overwrite what issued ones read, everybody else waits for their commit;
* at the end all loads and commits have arrived.
"""
import random

import pytest


class Machine:
    def __init__(self, counts, need):
        self.counts, self.need = counts, need      # arrivals per phase of a barrier; readers of a content
        self.arrived, self.done = {}, {}
        self.held = {}                             # buffer -> [content, landed, issued reads, done reads]
        self.loads, self.commits = [], []          # in flight
        self.open = []                             # products' effects that no commit tracks yet

    def arrive(self, bar):
        n = self.arrived.get(bar, 0) + 1
        if n == self.counts.get(bar, 1):
            n, self.done[bar] = 0, self.done.get(bar, 0) + 1
        self.arrived[bar] = n

    def replace(self, buf, what, landed, in_order):
        old = self.held.get(buf)
        if old is not None:
            assert old[2 if in_order else 3] == self.need(buf, old[0]), f"{buf}: {old[0]} overwritten by {what} early"
            assert in_order or old[1], f"{buf}: {old[0]} overwritten by {what} before it arrived"
        self.held[buf] = [what, landed, 0, 0]
        return self.held[buf]

    def read(self, buf, what, by_product):
        cell = self.held.get(buf)
        assert cell is not None and cell[0] == what, f"{buf} holds {cell}, {what} wanted"
        assert cell[1] is True or (by_product and cell[1] == "product"), f"{buf}: {what} read before it arrived"
        cell[2] += 1
        return cell

    def step(self, op):
        kind = op[0]
        if kind == "arrive":
            self.arrive(op[1])
        elif kind == "load":                       # buffer, content, barrier
            self.loads.append((self.replace(op[1], op[2], False, False), op[3]))
        elif kind == "put":
            self.replace(op[1], op[2], True, False)
        elif kind == "get":
            self.read(op[1], op[2], False)[3] += 1
        elif kind == "mma":                        # reads, writes
            for buf, what in op[1]:
                self.open.append(("read", self.read(buf, what, True)))
            for buf, what in op[2]:
                self.open.append(("write", self.replace(buf, what, "product", True)))
        elif kind == "commit":
            self.commits.append((self.open, op[1]))
            self.open = []

    def land(self, rng):
        """One load (any) or the oldest commit arrives."""
        if self.loads and (not self.commits or rng.random() < 0.5):
            cell, bar = self.loads.pop(rng.randrange(len(self.loads)))
            cell[1] = True
        else:
            effects, bar = self.commits.pop(0)
            for what, cell in effects:
                if what == "read":
                    cell[3] += 1
                elif cell[1] == "product":
                    cell[1] = True
        self.arrive(bar)


def simulate(roles, counts, need, seed):
    rng = random.Random(seed)
    m = Machine(counts, need)
    pending = {n: next(g, None) for n, g in roles.items()}
    land_p = (0.02, 0.2, 0.6)[seed % 3]
    favour = rng.choice(list(roles)) if seed % 2 else None        # one role runs whenever it can
    while any(pending.values()) or m.loads or m.commits:
        ready = []
        for n, op in pending.items():
            if op is None:
                continue
            if op[0] == "wait":
                c = m.done.get(op[1], 0)
                assert c <= op[2] + 1, f"{n}: wait on {op[1]} phase {op[2]} would alias (completed {c})"
                if c <= op[2]:
                    continue
            ready.append(n)
        flying = m.loads or m.commits
        assert ready or flying, "deadlock: " + str({n: op for n, op in pending.items() if op})
        if flying and (not ready or rng.random() < land_p):
            m.land(rng)
            continue
        n = favour if favour in ready else rng.choice(ready)
        m.step(pending[n])
        pending[n] = next(roles[n], None)
    return m


X = [("X", w, h) for w in range(2) for h in range(2)]      # score quarters: warpgroup, half
Y = [("Y", w, h) for w in range(2) for h in range(2)]


def put_all(region, what):
    return [(b, what) for b in region]


# ------------------------------------------------------------------ backward, dK and dV
def fixer(T, first, second, stages, ready):
    """Warp 2 where ranges are shorter than a tile: rewrites each tile (modelled as for every one)."""
    for j in range(T):
        for name, n in ((first, stages[0]), (second, stages[1])):
            s = j % n
            yield ("wait", f"{name}_FULL{s}", j // n)
            yield ("get", f"{name}{s}", (name, j))
            yield ("put", f"{name}{s}", (ready[name], j))
            yield ("arrive", f"{name}_FIXED{s}")


def with_fixer(roles, need, T, first, second, stages):
    """The same roles when warp 2 stands between the loads and the issuer."""
    ready = {first: first + "*", second: second + "*"}

    def issuer(ops):
        for op in ops:
            if op[0] == "wait" and op[1][:-1] in (f"{first}_FULL", f"{second}_FULL"):
                op = ("wait", op[1].replace("FULL", "FIXED"), op[2])
            elif op[0] == "mma":
                op = ("mma", [(b, (ready[w[0]], w[1])) if w[0] in ready and isinstance(w, tuple) else (b, w) for b, w in op[1]], op[2])
            yield op
    roles = dict(roles, issuer=issuer(roles["issuer"]), fixer=fixer(T, first, second, stages, ready))
    base = dict(need, **{ready[n]: need[n] for n in ready}, **{first: 1, second: 1})
    return roles, lambda buf, what: base[what[0]]


def kv_roles(T, q_stages=3, o_stages=2, shorts=False):
    def producer():
        yield ("load", "K", "K", "KV_FULL")
        yield ("load", "V", "V", "KV_FULL")
        for j in range(T):
            s, u = j % q_stages, j % o_stages
            if j >= q_stages:
                yield ("wait", f"Q_EMPTY{s}", j // q_stages - 1)
            yield ("load", f"Q{s}", ("Q", j), f"Q_FULL{s}")
            if j >= o_stages:
                yield ("wait", f"O_EMPTY{u}", j // o_stages - 1)
            yield ("load", f"O{u}", ("O", j), f"O_FULL{u}")

    def issuer():
        yield ("wait", "KV_FULL", 0)
        yield ("wait", "Q_FULL0", 0)
        yield ("wait", "O_FULL0", 0)
        yield ("mma", [("K", "K"), ("Q0", ("Q", 0))], put_all(X, ("S", 0)))
        yield ("commit", "S_FULL")
        yield ("mma", [("V", "V"), ("O0", ("O", 0))], put_all(Y, ("dP", 0)))
        yield ("commit", "DP_FULL")
        for j in range(T):
            s, u, s1, u1 = j % q_stages, j % o_stages, (j + 1) % q_stages, (j + 1) % o_stages
            more = j + 1 < T
            if more:
                yield ("wait", f"Q_FULL{s1}", (j + 1) // q_stages)
                yield ("wait", f"O_FULL{u1}", (j + 1) // o_stages)
            yield ("wait", "P_LO", j)
            yield ("mma", [(X[0], ("P", j)), (X[2], ("P", j)), (f"O{u}", ("O", j))], [])
            yield ("wait", "P_HI", j)
            yield ("mma", [(X[1], ("P", j)), (X[3], ("P", j)), (f"O{u}", ("O", j))], [])
            yield ("commit", f"O_EMPTY{u}")
            if more:
                yield ("mma", [("K", "K"), (f"Q{s1}", ("Q", j + 1))], put_all(X, ("S", j + 1)))
                yield ("commit", "S_FULL")
            yield ("wait", "DS_FULL", j)
            yield ("mma", [(b, ("dS", j)) for b in Y] + [(f"Q{s}", ("Q", j))], [])
            yield ("commit", f"Q_EMPTY{s}")
            if more:
                yield ("mma", [("V", "V"), (f"O{u1}", ("O", j + 1))], put_all(Y, ("dP", j + 1)))
                yield ("commit", "DP_FULL")
            else:
                yield ("commit", "FINAL")

    def terms():
        for j in range(T):
            if j >= 2:
                yield ("wait", f"STAT_EMPTY{j & 1}", j // 2 - 1)
            yield ("put", f"STAT{j & 1}", ("T", j))
            yield ("arrive", f"STAT_FULL{j & 1}")

    def threads(w):
        for j in range(T):
            yield ("wait", f"STAT_FULL{j & 1}", j // 2)
            yield ("wait", "S_FULL", j)
            for h in range(2):
                yield ("get", ("X", w, h), ("S", j))
            for h, bar in ((0, "P_LO"), (1, "P_HI")):
                yield ("put", ("X", w, h), ("P", j))
                yield ("arrive", bar)
            yield ("wait", "DP_FULL", j)
            for h in range(2):
                yield ("get", ("Y", w, h), ("dP", j))
            yield ("get", f"STAT{j & 1}", ("T", j))
            for h in range(2):
                yield ("put", ("Y", w, h), ("dS", j))
            yield ("arrive", "DS_FULL")
            yield ("arrive", f"STAT_EMPTY{j & 1}")
        yield ("wait", "FINAL", 0)

    counts = {"KV_FULL": 2, "P_LO": 2, "P_HI": 2, "DS_FULL": 2, "STAT_EMPTY0": 2, "STAT_EMPTY1": 2}
    need = {"Q": 2, "O": 3, "S": 1, "P": 1, "dP": 1, "dS": 1, "T": 2}
    roles = dict(producer=producer(), issuer=issuer(), terms=terms(), wg0=threads(0), wg1=threads(1))
    if shorts:
        roles, needs = with_fixer(roles, need, T, "Q", "O", (q_stages, o_stages))
        return roles, counts, needs
    return roles, counts, lambda buf, what: need[what[0]]


# ------------------------------------------------------------------ backward, dQ
def q_roles(T, k_stages=3, v_stages=2, shorts=False):
    def region(i):
        return [(f"R{i % 3}", w) for w in range(2)]

    def producer():
        yield ("load", "Q", "Q", "OWN_FULL")
        yield ("load", "dO", "dO", "OWN_FULL")
        for j in range(T):
            s, u = j % k_stages, j % v_stages
            if j >= k_stages:
                yield ("wait", f"K_EMPTY{s}", j // k_stages - 1)
            yield ("load", f"K{s}", ("K", j), f"K_FULL{s}")
            if j >= v_stages:
                yield ("wait", f"V_EMPTY{u}", j // v_stages - 1)
            yield ("load", f"V{u}", ("V", j), f"V_FULL{u}")

    def score(j):
        return ("mma", [("Q", "Q"), (f"K{j % k_stages}", ("K", j))], put_all(region(2 * j), ("S", j)))

    def issuer():
        yield ("wait", "OWN_FULL", 0)
        yield ("wait", "K_FULL0", 0)
        yield ("wait", "V_FULL0", 0)
        if T > 1:
            yield ("wait", "K_FULL1", 0)
        yield score(0)
        yield ("commit", "S_FULL0")
        yield ("mma", [("dO", "dO"), ("V0", ("V", 0))], put_all(region(1), ("dP", 0)))
        yield ("commit", "V_EMPTY0")
        yield ("commit", "DP_FULL0")
        if T > 1:
            yield score(1)
            yield ("commit", "S_FULL1")
        for j in range(T):
            b = j & 1
            if j + 1 < T:
                yield ("wait", f"V_FULL{b ^ 1}", (j + 1) // v_stages)
                yield ("wait", f"S_READ{b}", j // 2)
                yield ("mma", [("dO", "dO"), (f"V{b ^ 1}", ("V", j + 1))], put_all(region(2 * j), ("dP", j + 1)))
                yield ("commit", f"V_EMPTY{b ^ 1}")
                yield ("commit", f"DP_FULL{b ^ 1}")
            yield ("wait", f"DS_FULL{b}", j // 2)
            yield ("mma", [(x, ("dS", j)) for x in region(2 * j + 1)] + [(f"K{j % k_stages}", ("K", j))], [])
            yield ("commit", f"K_EMPTY{j % k_stages}")
            if j + 2 < T:
                yield ("wait", f"K_FULL{(j + 2) % k_stages}", (j + 2) // k_stages)
                yield score(j + 2)
                yield ("commit", f"S_FULL{b}")
            if j + 1 == T:
                yield ("commit", "FINAL")

    def threads(w):
        for j in range(T):
            b = j & 1
            yield ("wait", f"S_FULL{b}", j // 2)
            yield ("get", region(2 * j)[w], ("S", j))
            yield ("arrive", f"S_READ{b}")
            yield ("wait", f"DP_FULL{b}", j // 2)
            yield ("get", region(2 * j + 1)[w], ("dP", j))
            yield ("put", region(2 * j + 1)[w], ("dS", j))
            yield ("arrive", f"DS_FULL{b}")
        yield ("wait", "FINAL", 0)

    counts = {"OWN_FULL": 2, **{f"{n}{b}": 2 for n in ("S_READ", "DS_FULL") for b in range(2)}}
    need = {"K": 2, "V": 1, "S": 1, "dP": 1, "dS": 1}
    roles = dict(producer=producer(), issuer=issuer(), wg0=threads(0), wg1=threads(1))
    if shorts:
        roles, needs = with_fixer(roles, need, T, "K", "V", (k_stages, v_stages))
        return roles, counts, needs
    return roles, counts, lambda buf, what: need[what[0]]


# ------------------------------------------------------------------ attention over the cache
def cache_roles(T, nx, stages=2):
    """nx query tiles.  A score region is two halves, which P is handed over in; O leaves over Q."""
    def loader():
        for x in range(nx):
            yield ("load", f"Q{x}", "Q", "Q_FULL")

    def score(x, j):
        return ("mma", [(f"Q{x}", "Q"), (f"K{j % stages}", ("K", j))], [((f"S{x}", h), ("S", j)) for h in range(2)])

    def issuer():
        yield ("wait", "Q_FULL", 0)
        yield ("wait", "K_FULL0", 0)
        for x in range(nx):
            yield score(x, 0)
            yield ("commit", f"S_FULL{x}")
        yield ("commit", "K_EMPTY0")
        yield ("wait", "V_FULL0", 0)
        for j in range(T):
            s, s1, more = j % stages, (j + 1) % stages, j + 1 < T
            for x in range(nx):
                yield ("wait", f"P_LO{x}", j)
                yield ("mma", [((f"S{x}", 0), ("P", j)), (f"V{s}", ("V", j))], [])
                if more and x == 0:
                    yield ("wait", f"K_FULL{s1}", (j + 1) // stages)
                if more and x == nx - 1:
                    yield ("wait", f"V_FULL{s1}", (j + 1) // stages)
                yield ("wait", f"P_HI{x}", j)
                yield ("mma", [((f"S{x}", 1), ("P", j)), (f"V{s}", ("V", j))], [])
                if not more:
                    yield ("commit", f"O_FINAL{x}")
                if x == nx - 1:
                    yield ("commit", f"V_EMPTY{s}")
                if more:
                    yield score(x, j + 1)
                    yield ("commit", f"S_FULL{x}")
                    if x == nx - 1:
                        yield ("commit", f"K_EMPTY{s1}")

    def softmax(x):
        for j in range(T):
            yield ("wait", f"S_FULL{x}", j)
            for h in range(2):
                yield ("get", (f"S{x}", h), ("S", j))
            for h, bar in ((0, "P_LO"), (1, "P_HI")):
                yield ("put", (f"S{x}", h), ("P", j))
                yield ("arrive", f"{bar}{x}")
        yield ("wait", f"O_FINAL{x}", 0)
        yield ("put", f"Q{x}", "O")

    def widen():
        for j in range(T):
            s = j % stages
            for kv in "KV":
                if j >= stages:
                    yield ("wait", f"{kv}_EMPTY{s}", j // stages - 1)
                yield ("put", f"{kv}{s}", (kv, j))
                yield ("arrive", f"{kv}_FULL{s}")

    need = {"K": nx, "V": 2 * nx, "S": 1, "P": 1, "Q": T}
    roles = dict(loader=loader(), issuer=issuer(), widen=widen(), **{f"softmax{x}": softmax(x) for x in range(nx)})
    return roles, {"Q_FULL": nx}, lambda buf, what: need[what[0]]


@pytest.mark.parametrize("T", list(range(1, 20)))
@pytest.mark.parametrize("kind", ["kv", "q", "kv-short", "q-short", "cache1", "cache2"])
def test_protocol(kind, T):
    for seed in range(20):
        roles, counts, need = {"kv": lambda: kv_roles(T), "q": lambda: q_roles(T), "kv-short": lambda: kv_roles(T, shorts=True),
                               "q-short": lambda: q_roles(T, shorts=True), "cache1": lambda: cache_roles(T, 1),
                               "cache2": lambda: cache_roles(T, 2)}[kind]()
        m = simulate(roles, counts, need, seed)
        assert not m.open


def test_the_model_notices_a_missing_wait_and_a_missing_stage():
    def without(roles, name, skip):
        roles = dict(roles)
        roles[name] = (op for op in roles[name] if op[:2] != skip)
        return roles

    for make, name, skip in [(lambda: kv_roles(9), "issuer", ("wait", "DS_FULL")), (lambda: q_roles(9), "issuer", ("wait", "S_READ0")),
                             (lambda: cache_roles(9, 2), "widen", ("wait", "K_EMPTY0")), (lambda: kv_roles(9), "wg0", ("wait", "DP_FULL"))]:
        with pytest.raises(AssertionError):
            for seed in range(20):
                roles, counts, need = make()
                simulate(without(roles, name, skip), counts, need, seed)
