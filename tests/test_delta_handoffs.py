"""CPU proof of the hand-offs in the gated delta rule's sweeps (csrc/la_delta_tc.cu), by what
happens before what: every role's waits, arrivals and accesses of a chunk, in program order, as a
graph.  An mbarrier's wait goes by its phase's parity, so two things have to hold whatever the
warps' speeds are:

  * phase k + 1 of a barrier completes only after every wait for phase k has been passed (a waiter
    that comes later would take phase k + 1 for the one before and wait for good);
  * two accesses of one place, one of them a write, are in order.

The roles: the loads, the warp that issues the products, the tensor pipe (which does them in
order), two warps of the chain, two of each kind of the side warps, the stores.
"""
import itertools
import os
import re

import pytest

NS, NT = 2, 4
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "linear_attention_head_gb300", "csrc", "la_delta_tc.cu")
CHAIN, SIDE_P, SIDE_Q = ("chain0", "chain1"), ("sideP0", "sideP1"), ("sideQ0", "sideQ1")
SIDE = SIDE_P + SIDE_Q


class Graph:
    def __init__(self):
        self.edges, self.label = [], []     # successors of a node
        self.arrivals, self.waits, self.access = {}, [], []
        self.last = {}                      # a role's last node

    def node(self, label, *after):
        self.edges.append([])
        self.label.append(label)
        for a in after:
            if a is not None:
                self.edges[a].append(len(self.edges) - 1)
        return len(self.edges) - 1

    def step(self, role, label):
        self.last[role] = self.node((role, label), self.last.get(role))
        return self.last[role]

    def wait(self, role, bar, phase):
        self.waits.append((self.step(role, "wait %s %d" % (bar, phase)), bar, phase))

    def arrive(self, role, bar, phase):
        self.arrivals.setdefault((bar, phase), []).append(self.step(role, "arrive " + bar))

    def touch(self, role, write, *places):
        """Places: (name, part); part None is all of it."""
        n = self.step(role, "access")
        self.access += [(n, write, p if isinstance(p, tuple) else (p, None)) for p in places]
        return n

    def load(self, role, place, bar, phase):
        """An asynchronous copy: after what the role has done, done when its barrier is."""
        n = self.node(("copy", bar), self.step(role, "ask"))
        self.access.append((n, True, (place, None)))
        self.arrivals.setdefault((bar, phase), []).append(n)

    def close(self):
        """Barriers' completions as nodes; reachability."""
        done = {key: self.node(("phase",) + key, *nodes) for key, nodes in self.arrivals.items()}
        for n, bar, phase in self.waits:
            assert (bar, phase) in done, "nobody completes %s %d" % (bar, phase)
            self.edges[done[bar, phase]].append(n)
        for (bar, phase), n in done.items():
            if phase:
                self.edges[done[bar, phase - 1]].append(n)
        order, left = [], [0] * len(self.edges)
        for e in self.edges:
            for b in e:
                left[b] += 1
        free = [n for n, x in enumerate(left) if x == 0]
        while free:
            n = free.pop()
            order.append(n)
            for b in self.edges[n]:
                left[b] -= 1
                if left[b] == 0:
                    free.append(b)
        assert len(order) == len(self.edges), "waits in a circle"
        self.reach = [0] * len(self.edges)      # bit sets
        for n in reversed(order):
            r = 1 << n
            for b in self.edges[n]:
                r |= self.reach[b]
            self.reach[n] = r
        return done

    def before(self, a, b):
        return bool(self.reach[a] >> b & 1)


def sweep(bwd, keep, states, some_o, nc, turns):
    """The graph of nc chunks.  turns: how many barriers take turns (td_ready, e_ready, e_free)."""
    g = Graph()
    n_td, n_er, n_ef = turns
    of = lambda name, n, c: ("%s[%d]" % (name, c % n), c // n)
    stage = lambda name, c: "%s[%d]" % (name, c % NS)

    def product(label, writes, *reads):
        """Issued by its warp, done in order by the pipe."""
        issue = g.step("products", label)
        n = g.touch("pipe", False, *reads)
        g.edges[issue].append(n)
        g.access += [(n, True, (w, None)) for w in writes]

    def commit(bar, phase):
        issue = g.step("products", "commit " + bar)
        g.arrive("pipe", bar, phase)
        g.edges[issue].append(g.last["pipe"])

    # loads
    tables = 0
    for c in range(nc):
        while tables < nc and tables < c + 2:
            if tables >= NT:
                g.wait("loads", "tempty[%d]" % (tables % NT), tables // NT - 1)
            g.load("loads", "TAB[%d]" % (tables % NT), "tfull[%d]" % (tables % NT), tables // NT)
            tables += 1
        if c >= NS:
            if keep:
                g.wait("loads", *of("e_free", n_ef, c - NS))
            g.wait("loads", stage("empty", c), c // NS - 1)
        for place, bar in (("Q", "full"), ("K", "full"), ("VD", "fullv"), ("BB", "fullb")):
            g.load("loads", stage(place, c), stage(bar, c), c // NS)

    # products
    mma = "products"

    def stage_in(c):
        g.wait(mma, stage("full", c), c // NS)
        g.wait(mma, stage("fullb", c), c // NS)

    def scores(c):
        product("scores", ["T2" if bwd else "TR"], stage("Q", c), stage("K", c))
        commit("sc_full", c)

    def prior(c):
        g.wait(mma, "p_ready", c)
        g.wait(mma, *of("td_ready", n_td, c))
        product("prior", ["T2"], "TD[%d]" % (c & 1), "P")

    def solve(c):
        product("solve", ["T1"], "TY", stage("BB", c))
        commit("e_full", c)

    def update(c):
        product("update", ["TS"], "TY", stage("K", c))
        commit("s_full", c)
        commit(stage("empty", c), c // NS)

    stage_in(0)
    if bwd:
        scores(0)
        prior(0)
    for c in range(nc):
        g.wait(mma, "s_ready", c)
        product("K S", ["T1"], "TSH", stage("K", c))
        commit("ks_full", c)
        if bwd:
            g.wait(mma, "q_ready", c)
            product("Q dO", ["TS"], "TD[%d]" % (c & 1), "QOFF")
        elif not states:
            if c:
                g.wait(mma, "q_ready", c - 1)
                g.wait(mma, "r_ready", c - 1)
            product("Q S", ["T2"], "TSH", stage("Q", c))
            scores(c)
        g.wait(mma, "y_ready", c)
        solve(c)
        if c + 1 < nc:
            stage_in(c + 1)
            if bwd:
                scores(c + 1)
        g.wait(mma, "w_ready", c)
        update(c)
        if bwd:
            if c + 1 < nc:
                prior(c + 1)
        elif not states:
            g.wait(mma, "p_ready", c)
            g.wait(mma, "d_ready", c)
            product("P Eps", ["TR"], "T1", "P")
            commit("o_full", c)

    commit("drain", 0)
    g.wait(mma, "drain", 0)

    # chain
    for w in CHAIN:
        for c in range(nc):
            g.wait(w, "tfull[%d]" % (c % NT), c // NT)
            if c:
                g.wait(w, "s_full", c - 1)
            g.touch(w, False, "TAB[%d]" % (c % NT))
            g.touch(w, True, ("TS", w), ("TSH", w))
            g.arrive(w, "s_ready", c)
            if keep:
                if c:
                    g.wait(w, "i_free", c - 1)
                g.touch(w, False, ("TSH", w))
                g.touch(w, True, ("SOFF", w))
                g.arrive(w, "i_ready", c)
            if not bwd:
                g.wait(w, stage("fullv", c), c // NS)
                g.touch(w, False, stage("VD", c))
            g.wait(w, "ks_full", c)
            if bwd:
                g.touch(w, False, ("T2", w))
            g.touch(w, True, ("T1", w), ("TY", w))
            g.arrive(w, "y_ready", c)
            g.wait(w, "e_full", c)
            g.touch(w, False, ("T1", w))
            g.touch(w, True, ("TY", w))
            g.arrive(w, "w_ready", c)
            if bwd and keep:    # R's image, and dV's
                g.touch(w, True, (stage("VD", c), w), (stage("Q", c), w))
                g.arrive(w, *of("e_ready", n_er, c))
            if not bwd and not states:
                if keep:
                    g.wait(w, "x_read", c)
                g.touch(w, True, ("T1", w))
                g.arrive(w, "d_ready", c)
            g.touch(w, False, "TAB[%d]" % (c % NT))
            g.arrive(w, "tempty[%d]" % (c % NT), c // NT)
        g.wait(w, "s_full", nc - 1)
        g.touch(w, False, ("TS", w))

    # side
    for w in SIDE if bwd or not states else ():
        for c in range(nc):
            if bwd:
                g.wait(w, stage("fullv", c), c // NS)
                g.touch(w, False, stage("VD", c))
                g.touch(w, True, ("TD[%d]" % (c & 1), w))
                g.arrive(w, *of("td_ready", n_td, c))
            g.wait(w, "tfull[%d]" % (c % NT), c // NT)
            g.wait(w, "sc_full", c)
            g.touch(w, False, "TAB[%d]" % (c % NT))
            if w in SIDE_P:
                g.touch(w, False, "T2" if bwd else "TR")
                g.touch(w, True, ("P", w))
                g.arrive(w, "p_ready", c)
            elif bwd:
                g.wait(w, stage("full", c), c // NS)
                g.touch(w, False, stage("Q", c))
                g.touch(w, True, ("QOFF", w))
                g.arrive(w, "q_ready", c)
            if not bwd:
                if keep:
                    g.wait(w, "e_full", c)
                    g.touch(w, False, "T1")
                    g.arrive(w, "x_read", c)
                    g.touch(w, True, (stage("VD", c), w))
                    g.arrive(w, *of("e_ready", n_er, c))
                g.touch(w, False, "T2")
                g.arrive(w, "q_ready", c)
                g.wait(w, "o_full", c)
                g.touch(w, False, "TR")
                g.arrive(w, "r_ready", c)
                if some_o:
                    if c:
                        g.wait(w, "o_free", c - 1)
                    g.touch(w, True, ("OOFF", w))
                    g.arrive(w, "o_ready", c)
            g.touch(w, False, "TAB[%d]" % (c % NT))
            g.arrive(w, "tempty[%d]" % (c % NT), c // NT)

    # stores (each waits until its source has been read)
    for c in range(nc):
        if keep:
            g.wait("stores", "i_ready", c)
            g.touch("stores", False, "SOFF")
            g.arrive("stores", "i_free", c)
            g.wait("stores", *of("e_ready", n_er, c))
            g.touch("stores", False, stage("VD", c), *([stage("Q", c)] if bwd else []))
            g.arrive("stores", *of("e_free", n_ef, c))
        if some_o:
            g.wait("stores", "o_ready", c)
            g.touch("stores", False, "OOFF")
            g.arrive("stores", "o_free", c)
    return g


def faults(g):
    """(barriers a waiter can miss a phase of, places with accesses in no order)"""
    done = g.close()
    missed = {re.sub(r"\[.*", "", bar) for n, bar, phase in g.waits
              if (bar, phase + 1) in done and not g.before(n, done[bar, phase + 1])}
    places = {}
    for n, write, (name, part) in g.access:
        places.setdefault(name, []).append((n, write, part))
    unordered = set()
    for name, xs in places.items():
        for (a, wa, pa), (b, wb, pb) in itertools.combinations(xs, 2):
            if a != b and (wa or wb) and (pa is None or pb is None or pa == pb) and \
                    not g.before(a, b) and not g.before(b, a):
                unordered.add(name)
    return missed, unordered


# backward, images kept, states alone, O wanted
MODES = [(False, False, False, True), (False, True, False, True), (False, True, False, False),
         (False, False, True, False), (True, True, False, False), (True, False, True, False)]


@pytest.mark.parametrize("nc", [1, 2, 3, 9])
@pytest.mark.parametrize("mode", MODES)
def test_no_phase_is_missed(mode, nc):
    assert faults(sweep(*mode, nc, turns=(2, NS, NS))) == (set(), set())


def test_one_barrier_for_both_stages_can_be_missed():
    # what turns are there for: with a single barrier each, a late waiter misses a phase
    assert faults(sweep(False, True, False, True, 9, turns=(1, 1, 1)))[0] == {"e_ready", "e_free"}
    assert faults(sweep(True, True, False, False, 9, turns=(1, 1, 1)))[0] == \
        {"td_ready", "e_ready", "e_free"}
    assert faults(sweep(True, True, False, False, 9, turns=(1, NS, NS)))[0] == {"td_ready"}
    assert faults(sweep(True, True, False, False, 9, turns=(2, 1, NS)))[0] == {"e_ready"}
    assert faults(sweep(True, True, False, False, 9, turns=(2, NS, 1)))[0] == {"e_free"}


def unclocked(g, drain):
    """Barriers that the chain or the side warps wait for although no wait with a clock (of the
    other roles; the last products' where drain is set) would run out if an arrival at them
    never came."""
    g.close()
    clocked = [n for n, bar, _ in g.waits
               if g.label[n][0] in ("loads", "products", "stores") and (drain or bar != "drain")]
    return {bar for n, bar, phase in g.waits if g.label[n][0] in CHAIN + SIDE
            for a in g.arrivals[bar, phase] if not any(g.before(a, c) for c in clocked)}


@pytest.mark.parametrize("nc", [1, 2, 9])
@pytest.mark.parametrize("mode", MODES)
def test_every_wait_ends(mode, nc):
    g = sweep(*mode, nc, turns=(2, NS, NS))
    assert unclocked(g, True) == set()
    # what the last products' wait is needed for: where no O goes to the stores' waits
    assert ("s_full" in unclocked(g, False)) == (not mode[3])


def test_the_last_products_raise_the_flag():
    with open(SOURCE) as f:
        text = f.read()
    assert re.search(r"drain_wait\(drain, 0\);\s+if \(!mbar_try_wait\(drain, 0\)\)[^\n]*\n"
                     r"\s+\*abort_flag = 1;", text)


def test_the_kernel_has_these_barriers():
    with open(SOURCE) as f:
        text = f.read()
    # those that take turns: waited for and arrived at by stage (by chunk's parity)
    for name, uses in (("td_ready", 2), ("e_ready", 3), ("e_free", 2)):
        assert len(re.findall(r"&%s\[" % name, text)) >= uses, name
        assert not re.search(r"(wait_\w+(<BWD>)?|both|mbar_arrive)\(%s\b" % name, text), name
    # the model knows every barrier of the sweep
    names = set(re.findall(r"uint64_t \*(\w+) = bars", text)) - {"in_full"}
    model = set()
    for mode in MODES:
        model |= {re.sub(r"\[.*", "", bar) for bar, _ in sweep(*mode, 3, (2, NS, NS)).arrivals}
    ring = {"full", "fullv", "fullb", "empty", "tfull", "tempty"}
    assert names <= model and model - names <= ring | {"e_free"}, names ^ model
