"""The barriers of the tcgen05 attention kernel (kv8_wide.cu), proved on a model of its warps (CPU).

Each warp, the tensor core and every bulk copy is a list of steps: wait for a phase of an mbarrier entry, arrive on one,
read or write a buffer.  A wait sees an entry's parity alone, so it is right only if, in every order of the steps,
  (a) the phase before the one it means is known to be complete (else it passes too early), and
  (b) the phase after it cannot complete before it has passed (else the parity is back and it may wait for ever).
An arrival has to know that its entry's earlier phases are complete (else it counts for one of those).  All three, and the
order of every two accesses of a buffer, are read off vector clocks: what a step knows to have happened.  The clocks
do not depend on the order in which the model takes the steps, so one pass speaks for all orders.

Depths and arrival counts are taken from the source.
"""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a8_verify_gb300", "csrc",
                   "kv8_wide.cu")


def _source():
    return re.sub(r"//[^\n]*", "", open(SRC).read())


def _constants(text):
    """Warp numbers, ring depths, entries of each barrier."""
    k = {n: int(v) for n, v in re.findall(r"\b(k\w+) = (\d+)[,;]", text)}
    bars = {}
    for name, size in re.findall(r"(\w+)(?:\[(\w+)\])?[,;]", re.search(r"struct Bars \{\s*uint64_t ([^}]*)\}", text).group(1)):
        bars[name] = 1 if not size else k[size] if size in k else int(size)
    return k, bars


class Model:
    def __init__(self, counts):
        self.counts = counts                     # arrivals of a phase, by barrier
        self.steps = {}                          # role -> [(kind, ...)]
        self.ends = []                           # (role, role that has to be done by its end)

    def add(self, role, *step):
        self.steps.setdefault(role, []).append(step)

    def check(self):
        """Runs every role to its end and returns what is wrong."""
        arrivals, waits, accesses, bad = {}, {}, {}, []
        clock = {r: {} for r in self.steps}      # role -> last step of every role known to be done
        at = dict.fromkeys(self.steps, 0)
        moved = True
        while moved:
            moved = False
            for r, steps in self.steps.items():
                while at[r] < len(steps):
                    kind, what, phase = steps[at[r]]
                    known = clock[r]
                    if kind == "wait":
                        got = arrivals.get((what, phase), [])
                        if len(got) < self.counts[what[0]]:
                            break
                        before = arrivals.get((what, phase - 1), []) if phase else []
                        if any(known.get(a, -1) < i for a, i, _ in before):
                            bad.append("%s: the wait for phase %d of %s may pass one phase early" % (r, phase, what))
                        for _, _, c in got:
                            for a, i in c.items():
                                known[a] = max(known.get(a, -1), i)
                        waits.setdefault((what, phase), []).append((r, at[r]))
                    elif kind == "arrive":
                        before = arrivals.get((what, phase - 1), []) if phase else []
                        if phase and (len(before) < self.counts[what[0]] or any(known.get(a, -1) < i for a, i, _ in before)):
                            bad.append("%s: the arrival of phase %d of %s may count for an earlier one" % (r, phase, what))
                    else:                        # a read or a write of buffer `what`
                        for a, i, write in accesses.get(what, []):
                            if a != r and (write or kind == "write") and known.get(a, -1) < i:
                                bad.append("%s: %s of %s races with %s" % (r, kind, what, a))
                        accesses.setdefault(what, []).append((r, at[r], kind == "write"))
                    known[r] = at[r]
                    if kind == "arrive":
                        arrivals.setdefault((what, phase), []).append((r, at[r], dict(known)))
                    at[r] += 1
                    moved = True
        for r, steps in self.steps.items():
            if at[r] < len(steps):
                bad.append("%s stops at %s" % (r, steps[at[r]]))
        for (what, phase), who in waits.items():
            after = arrivals.get((what, phase + 1), [])
            if len(after) < self.counts[what[0]]:
                continue
            for r, i in who:
                if all(c.get(r, -1) < i for _, _, c in after):
                    bad.append("%s: phase %d of %s may complete before its wait for phase %d" % (r, phase + 1, what, phase))
        for r, last in self.ends:                # what has to be done when a role ends
            if clock[r].get(last, -1) < len(self.steps[last]) - 1:
                bad.append("%s ends before %s" % (r, last))
        return bad


def wide_model(text, runs, fp32, vec):
    """The kernel's roles over a CTA's runs of pages."""
    k, bars = _constants(text)
    nq, np_, no = (2, 1, 1) if fp32 else (1, 2, 2)
    soft = ["soft%d" % w for w in range(k["kSoftWarps"])]
    sums = ["sum%d" % w for w in range(k["kSumWarps"])]
    convs = ["conv%d" % w for w in range(k["kConvWarps"])]
    half = len(convs) // 2
    m = Model(dict(code_full=1, code_empty=len(convs), k_full=half, v_full=half, s_done=1, pv_done=1, s_empty=len(soft),
                   p_full=len(soft), o_empty=len(sums), lo_empty=len(soft), q_full=1, q_empty=len(soft), issue=1, drained=1))
    depth = dict(bars, o_empty=no)               # the products use NO of its entries

    def ev(role, kind, name, n):                 # the n-th use of a barrier: entry and phase
        d = depth[name]
        m.add(role, kind, (name, n % d), n // d)

    issued = [0]

    def tensor(reads, writes, commits):          # one batch of products: issued by its warp, done in order, committed
        m.add("mma", "arrive", ("issue", issued[0]), 0)
        m.add("tensor", "wait", ("issue", issued[0]), 0)
        issued[0] += 1
        for b in reads:
            m.add("tensor", "read", b, 0)
        for b in writes:
            m.add("tensor", "write", b, 0)
        for name, n in commits:
            ev("tensor", "arrive", name, n)

    total = sum(runs)
    # the copy warp and its copies
    for p in range(total):
        if p >= k["kRing"]:
            ev("copy", "wait", "code_empty", p - k["kRing"])
        m.add("copy", "arrive", ("issue", "code%d" % p), 0)
        m.add("code%d" % p, "wait", ("issue", "code%d" % p), 0)
        m.add("code%d" % p, "write", ("ring", p % k["kRing"]), 0)
        ev("code%d" % p, "arrive", "code_full", p)
    if vec:                                      # query rows come before their run's pages
        first, at, where = m.steps.pop("copy"), 0, 0
        m.steps["copy"] = []
        for i, pages in enumerate(runs):
            if i:
                ev("copy", "wait", "q_empty", i - 1)
            m.add("copy", "arrive", ("issue", "q%d" % i), 0)
            m.add("q%d" % i, "wait", ("issue", "q%d" % i), 0)
            m.add("q%d" % i, "write", ("rows",), 0)
            ev("q%d" % i, "arrive", "q_full", i)
            for p in range(at, at + pages):
                take = 2 if p >= k["kRing"] else 1
                m.steps["copy"] += first[where:where + take]
                where += take
            at += pages
    # converters
    for w, r in enumerate(convs):
        v = w // half
        for p in range(total):
            if p >= 2:
                ev(r, "wait", "pv_done" if v else "s_done", p - 2)
            ev(r, "wait", "code_full", p)
            m.add(r, "read", ("ring", p % k["kRing"]), 0)
            m.add(r, "write", ("v" if v else "k", p % 2, w), 0)
            ev(r, "arrive", "code_empty", p)
            ev(r, "arrive", "v_full" if v else "k_full", p)
    quads = range(len(soft))
    tiles = {v: [("v" if v else "k", w) for w in range(v * half, v * half + half)] for v in (0, 1)}

    def values(n):
        ev("mma", "wait", "p_full", n)
        ev("mma", "wait", "v_full", n)
        if n >= no:
            ev("mma", "wait", "o_empty", n - no)
        tensor([("p", n % np_, q) for q in quads] + [(t, n % 2, w) for t, w in tiles[1]],
               [("o", n % no, s) for s in sums], [("pv_done", n)])

    n = 0
    for pages in runs:                           # products
        for p in range(pages):
            ev("mma", "wait", "k_full", n)
            ev("mma", "wait", "s_empty", n)
            kt = [(t, n % 2, w) for t, w in tiles[0]]
            if nq == 2:
                tensor([("q", q) for q in quads] + kt, [("s", n % 2, q) for q in quads], [])
                ev("mma", "wait", "lo_empty", n)
                tensor([("q", q) for q in quads] + kt, [("lo", q) for q in quads], [("s_done", n)])
            else:
                tensor([("q", q) for q in quads] + kt, [("s", n % 2, q) for q in quads], [("s_done", n)])
            if p > 0:
                values(n - 1)
            n += 1
        values(n - 1)
    give_up(m, text, issued)
    for q, r in enumerate(soft):                 # softmax
        n = freed = 0
        for i, pages in enumerate(runs):
            if vec:
                ev(r, "wait", "q_full", i)
                m.add(r, "read", ("rows",), 0)
            m.add(r, "write", ("q", q), 0)
            if vec:
                ev(r, "arrive", "q_empty", i)
            for _ in range(2):
                if freed < n + pages:
                    ev(r, "arrive", "s_empty", freed)
                    freed += 1
            if nq == 2:
                ev(r, "arrive", "lo_empty", n)
            for p in range(pages):
                ev(r, "wait", "s_done", n)
                m.add(r, "read", ("s", n % 2, q), 0)
                if n >= np_:
                    ev(r, "wait", "pv_done", n - np_)
                if nq == 2:
                    m.add(r, "read", ("lo", q), 0)
                m.add(r, "write", ("p", n % np_, q), 0)
                m.add(r, "write", ("fac", n % k["kFac"], q), 0)
                ev(r, "arrive", "p_full", n)
                if freed < n + pages - p:
                    ev(r, "arrive", "s_empty", freed)
                    freed += 1
                if nq == 2 and p + 1 < pages:
                    ev(r, "arrive", "lo_empty", n + 1)
                n += 1
            ev(r, "wait", "pv_done", n - 1)
    for w, r in enumerate(sums):                 # values
        for n in range(total):
            ev(r, "wait", "p_full", n)
            ev(r, "wait", "pv_done", n)
            m.add(r, "read", ("fac", n % k["kFac"], w % 4), 0)
            m.add(r, "read", ("o", n % no, r), 0)
            ev(r, "arrive", "o_empty", n)
    return m


def give_up(m, text, issued):
    """The product warp's end, after its last wait or the first that ran out: the tensor core has to be done."""
    m.ends.append(("mma", "tensor"))
    if re.search(r"tc_commit\(elect_one\(\), &bar\.drained\);[^;]*mbar_wait\(&bar\.drained, 0[,)][^;]*;\s*asm volatile\(\"tcgen05\.dealloc", text):
        m.add("mma", "arrive", ("issue", issued[0]), 0)
        m.add("tensor", "wait", ("issue", issued[0]), 0)
        m.add("tensor", "arrive", ("drained", 0), 0)
        m.add("mma", "wait", ("drained", 0), 0)


RUNS = [[1], [2], [3], [4], [5], [10], [2, 4], [1, 3], [1, 1, 1, 1, 1, 1], [3, 1, 2, 1, 4], [35, 1, 9], [40]]


@pytest.mark.parametrize("vec", [True, False])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("runs", RUNS, ids=str)
def test_no_wait_can_be_overtaken(runs, fp32, vec):
    bad = wide_model(_source(), runs, fp32, vec).check()
    assert not bad, bad[:5]


def test_the_source_uses_the_depths_of_the_model():
    """Every use of a barrier goes by a ring position of that barrier's depth."""
    text = _source()
    k, bars = _constants(text)
    assert "NP = NQ == 2 ? 1 : 2" in text and "NO = sizeof(T) == 4 ? 1 : 2" in text and "NQ = sizeof(T) == 4 ? 2 : 1" in text
    turns = {}
    for depth, name in re.findall(r"Turn<(\w+)> (\w+(?:, \w+)*)(?:;|\()", text):
        for one in name.split(", "):
            turns.setdefault(one, set()).add(k[depth] if depth in k else depth)
    used = {}
    for name, index in re.findall(r"bar\.(\w+)\[(\w+)\.i\]", text):
        used.setdefault(name, set()).add(index)
    for name, ring in used.items():
        for one in ring:
            want = {"NO"} if name == "o_empty" else {bars[name], str(bars[name])}
            assert turns[one] <= want, (name, one, turns[one])
    assert used["p_full"] and not re.search(r"bar\.p_full\[(?!\w+\.i\]|i\])", text)


def test_the_model_sees_a_ring_that_is_too_short():
    """Planted in the model: two entries of p_full (wrong in bf16 calls alone), one round of row factors."""
    text = _source()
    short = re.sub(r"p_full\[\w+\]", "p_full[2]", text, count=1)
    assert any("may complete before its wait" in x and "p_full" in x for x in wide_model(short, [4], False, True).check())
    assert not wide_model(short, [10], True, True).check()
    short = re.sub(r"kFac = \d+", "kFac = 1", text)
    assert any("fac" in x for x in wide_model(short, [6], False, False).check())


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("left", range(0, 60, 7))
def test_no_product_is_under_way_when_a_wait_has_run_out(fp32, left):
    """The product warp stops at its `left`th wait, the others where that leaves them; the tensor core is done at its end."""
    m = wide_model(_source(), [9], fp32, True)
    keep, issued, n = [], [0], 0
    for step in m.steps["mma"]:
        if step[0] == "wait":
            if n == left or step[1][0] == "drained":
                break
            n += 1
        keep.append(step)
    stopped = Model(m.counts)
    stopped.steps = {r: list(s) for r, s in m.steps.items()}
    issued[0] = sum(s[0] == "arrive" for s in keep)
    stopped.steps["mma"] = keep
    steps, stopped.steps["tensor"] = m.steps["tensor"], []
    for step in steps:
        if step[0] == "wait" and step[1][1] == issued[0]:
            break
        stopped.steps["tensor"].append(step)
    give_up(stopped, _source(), issued)
    assert not [x for x in stopped.check() if "ends before" in x]


def test_tensor_memory_is_taken_when_the_kernel_in_front_is_done():
    """A CTA may start while the kernel in front runs; if it took tensor memory before that has ended, a CTA of that kernel on
    the same SM could wait for it while it waits for that kernel."""
    body = _source().split("k_kv8_wide(w4a8_kv8_cache c")[1]
    assert 0 < body.index("griddep_enter();") < body.index("tcgen05.alloc")
