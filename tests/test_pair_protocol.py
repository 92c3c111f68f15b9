"""The barrier protocol of the paged pair kernel (csrc/attention_pair.cu), run on
the CPU without a GPU: a cluster's roles as coroutines in random orders.

An mbarrier wait names one parity bit.  It passes while the barrier's present
phase has the other parity, so it tells two neighbouring phases apart and no
more: a role that comes to its wait after the producer has completed two phases
waits for a phase that may never come.  The kernel is right if nothing can
complete a second phase before a role has waited for the first.

The model takes the barriers' arrival counts, the indexes and parities of all
waits, and the index of the arrivals on pv_sent from the source, so that it
follows changes of these; the order of a role's steps is written out here.
Copies and matrix instructions finish at random times after they were issued (those
of one issuer in their order), and every buffer carries what it should hold, so
that an early overwrite shows as well as a wait that never ends.
"""
import os
import random
import re

import pytest

from conftest import ROOT

SOURCE = os.path.join(ROOT, "long_context_compressed_02_b200", "csrc", "attention_pair.cu")
TILE_BLOCKS, ITEMS, STAGES, K_STAGES = 4, 4, 4, 8


# ------------------------------------------------------------------ what the source says

def _expr(text):
    return compile(text.replace("/", "//").replace("x.items", "items").strip(), "<source>", "eval")


def _barrier(text):
    """'&name[index]' or 'name' -> (name, compiled index)."""
    name, index = re.fullmatch(r"&?(\w+)(?:\[([^\]]*)\])?", text.strip()).groups()
    return name, _expr(index or "0")


class Source:
    def __init__(self, text):
        for name, value in (("kTileBlocks", TILE_BLOCKS), ("kItems", ITEMS), ("kStages", STAGES), ("kKStages", K_STAGES)):
            assert re.search(rf"constexpr int {name} = {value};", text), f"the model was written for {name} = {value}"
        self.counts = {}
        for bar, count in re.findall(r"mbar_init\(([^,]+), (\d+)\)", text):
            self.counts[_barrier(bar)[0]] = int(count)
        # the roles' parts of the kernel, by the comment that opens each
        heads = ["items", "queries and K", "V", "patches", "S (CTA 0)", "PV (CTA 0)", "softmax"]
        at = [text.index(f"// ============================ {h}") for h in heads]
        parts = {h: text[a:b] for h, a, b in zip(heads, at, at[1:] + [len(text)])}
        parts["next_item"] = text[text.index("auto next_item"):at[0]]
        self.waits = {}          # (role, barrier) -> [(index, parity, first tile that waits)]
        for role, body in parts.items():
            for first, bar, parity in re.findall(r"(?:\(t < (\d+) \|\| )?wait_warp\((&?\w+(?:\[[^\]]*\])?), (.*?), abort_flag\)", body):
                name, index = _barrier(bar)
                self.waits.setdefault((role, name), []).append((index, _expr(parity), int(first or 0)))
        self.sent = _barrier(re.search(r"mbar_arrive\((&?pv_sent(?:\[[^\]]*\])?)\)", parts["PV (CTA 0)"]).group(1))[1]


# ------------------------------------------------------------------ one cluster

class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def arrive(self, n=1, tx=0):
        self.tx += tx
        self.pending -= n
        assert self.pending >= 0, "more arrivals than the barrier counts"
        self.check()

    def copied(self, tx):
        self.tx -= tx
        self.check()

    def check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count


class Group:
    """A named barrier of n parties."""

    def __init__(self, n):
        self.n, self.here, self.round = n, 0, 0

    def join(self):
        mine = self.round
        self.here += 1
        if self.here == self.n:
            self.here, self.round = 0, self.round + 1
        return lambda: self.round > mine


class Cluster:
    """items: a list per item of its blocks, each clean (True) or to be patched."""

    GROUPS = 2                   # softmax parties of a CTA, 4 warps each

    def __init__(self, src, items, rng):
        self.src, self.items, self.rng = src, items, rng
        sizes = dict(full_k=STAGES, full_v=STAGES, empty_k=STAGES, empty_v=STAGES, patch=STAGES, w_full=ITEMS, w_free=ITEMS,
                     s_full=2, s_free=2, pv_sent=2)
        self.bars = [{name: [Bar(c) for _ in range(sizes.get(name, 1))] for name, c in src.counts.items()} for _ in range(2)]
        self.queues = {}         # issuer -> work that finishes in order
        self.done = [[] for _ in range(2 * self.GROUPS)]
        # contents: what a buffer holds, and operations that still read it
        self.ring = [[None] * ITEMS for _ in range(2)]
        self.q = [[None, 0] for _ in range(2)]
        self.k = [[[None, 0] for _ in range(STAGES)] for _ in range(2)]
        self.v = [[[None, 0] for _ in range(STAGES)] for _ in range(2)]
        self.s = [[None, 2 * self.GROUPS] for _ in range(2)]        # tile, readers that are through
        self.p = [[None] * self.GROUPS for _ in range(2)]
        self.o_read = 2 * self.GROUPS            # readers of the last item's output that are through
        self.o_tile = None

    # a wait as the source has it; every name that its expressions use is in `env`
    def wait(self, cta, role, name, which=0, **env):
        index, parity, first = self.src.waits[(role, name)][which]
        if env.get("t", 0) < first:
            return lambda: True
        env.update(kItems=ITEMS, kStages=STAGES)
        bar, par = self.bars[cta][name][eval(index, {}, env)], eval(parity, {}, env)
        return lambda: (bar.phase & 1) != par

    def later(self, issuer, fn):
        self.queues.setdefault(issuer, []).append(fn)

    def copy(self, fn):
        self.later(("copy", len(self.queues), self.rng.random()), fn)

    def tiles(self, item):
        return -(-len(item) // TILE_BLOCKS)

    # ---- shared by the roles
    def next_item(self, cta, k, arrivals, group=None):
        yield self.wait(cta, "next_item", "w_full", sl=k % ITEMS, k=k)
        if group:
            yield group.join()
        held, item = self.ring[cta][k % ITEMS]
        assert held == k, "an item was replaced before it was read"
        self.bars[cta]["w_free"][k % ITEMS].arrive(arrivals)
        return item

    def stream(self, cta, arrivals, group=None):
        """Yields waits, and ('tile', item, its number among those with tiles, tile) for each tile."""
        k = items = 0
        while True:
            item = yield from self.next_item(cta, k, arrivals, group)
            k += 1
            if item is None:
                return
            nt = self.tiles(item)
            items += nt > 0
            for i in range(nt):
                yield ("tile", item, items, i)

    # ---- the roles
    def role_items(self, cta):
        for k, item in enumerate(self.items + [None]):
            yield self.wait(cta, "items", "w_free", sl=k % ITEMS, k=k)
            self.ring[cta][k % ITEMS] = (k, item)
            self.bars[cta]["w_full"][k % ITEMS].arrive()

    def role_k(self, cta):
        st = t = 0
        for x in self.stream(cta, 1):
            if callable(x):
                yield x
                continue
            _, item, items, i = x
            if i == 0:
                yield self.wait(cta, "queries and K", "q_free", items=items)
                assert self.q[cta][1] == 0, "queries overwritten while products read them"
                self.bars[0]["q_full"][0].arrive(1, 1)
                self.q[cta][0] = None

                def land(items=items):
                    self.q[cta][0] = items
                    self.bars[0]["q_full"][0].copied(1)
                self.copy(land)
            n = max(0, min(2, min(TILE_BLOCKS, len(item) - TILE_BLOCKS * i) - 2 * cta))
            for d in range(K_STAGES):
                sl = st % STAGES
                yield self.wait(cta, "queries and K", "empty_k", sl=sl, st=st)
                assert self.k[cta][sl][1] == 0, "K overwritten while products read it"
                bar = self.bars[0]["full_k"][sl]
                bar.arrive(1, n)
                self.k[cta][sl][0] = None if n else (t, d)

                def land(sl=sl, tag=(t, d), n=n, bar=bar):
                    self.k[cta][sl][0] = tag
                    bar.copied(n)
                if n:
                    self.copy(land)
                st += 1
            t += 1

    def role_v(self, cta):
        st = t = 0
        for x in self.stream(cta, 1):
            if callable(x):
                yield x
                continue
            _, item, _, i = x
            blocks = item[TILE_BLOCKS * i:TILE_BLOCKS * (i + 1)]
            for v in range(2 * len(blocks)):
                sl = st % STAGES
                yield self.wait(cta, "V", "empty_v", sl=sl, st=st)
                assert self.v[cta][sl][1] == 0, "V overwritten while products read it"
                clean = blocks[v >> 1]
                bar = self.bars[0]["full_v"][sl] if clean else self.bars[cta]["patch"][sl]
                bar.arrive(1, 1)
                self.v[cta][sl][0] = None

                def land(sl=sl, tag=(t, v, clean), bar=bar):
                    self.v[cta][sl][0] = tag
                    bar.copied(1)
                self.copy(land)
                st += 1
            t += 1

    def role_patch(self, cta):
        st = t = uses = 0
        for x in self.stream(cta, 2):
            if callable(x):
                yield x
                continue
            _, item, _, i = x
            blocks = item[TILE_BLOCKS * i:TILE_BLOCKS * (i + 1)]
            for v in range(2 * len(blocks)):
                sl = st % STAGES
                st += 1
                if blocks[v >> 1]:
                    continue
                yield self.wait(cta, "patches", "patch", sl=sl, uses=uses)
                uses ^= 1 << sl
                assert self.v[cta][sl][0] == (t, v, False), "a patch of another block"
                self.v[cta][sl][0] = (t, v, True)
                self.bars[0]["full_v"][sl].arrive()
            t += 1

    def commit(self, issuer, name, index, reads=()):
        """Arrives in both CTAs once the issuer's products so far are done."""
        def fn():
            for r in reads:
                r[1] -= 1
            for c in range(2):
                self.bars[c][name][index].arrive()
        self.later(issuer, fn)

    def role_s(self, cta):
        st = t = 0
        for x in self.stream(cta, 1):
            if callable(x):
                yield x
                continue
            if cta != 0:
                continue
            _, item, items, i = x
            if i == 0:
                yield self.wait(0, "S (CTA 0)", "q_full", items=items)
            yield self.wait(0, "S (CTA 0)", "pv_sent", t=t)
            yield self.wait(0, "S (CTA 0)", "s_free", t=t)
            for c in range(2):
                assert self.q[c][0] == items, "products with the queries of another item"
                self.q[c][1] += 1
            assert self.s[t & 1][1] == 2 * self.GROUPS, "logits overwritten before they were read"
            self.s[t & 1] = [None, 0]
            for d in range(K_STAGES):
                sl = st % STAGES
                yield self.wait(0, "S (CTA 0)", "full_k", sl=sl, st=st)
                for c in range(2):
                    assert self.k[c][sl][0] == (t, d), "products with other keys"
                    self.k[c][sl][1] += 1
                self.commit("S", "empty_k", sl, [self.k[0][sl], self.k[1][sl]])
                st += 1

            def made(t=t):
                self.s[t & 1][0] = t
                for c in range(2):
                    self.q[c][1] -= 1
            self.later("S", made)
            self.commit("S", "s_full", t & 1)
            if i == self.tiles(item) - 1:
                self.commit("S", "q_free", 0)
            t += 1

    def role_pv(self, cta):
        st = t = 0
        for x in self.stream(cta, 1):
            if callable(x):
                yield x
                continue
            if cta != 0:
                continue
            _, item, items, i = x
            if i == 0:
                yield self.wait(0, "PV (CTA 0)", "o_free", items=items)
                assert self.o_read == 2 * self.GROUPS, "an output overwritten before it was read"
                self.o_read = 0
            yield self.wait(0, "PV (CTA 0)", "p_full", t=t)
            assert all(p == t for c in range(2) for p in self.p[c]), "products with other weights"
            for v in range(2 * min(TILE_BLOCKS, len(item) - TILE_BLOCKS * i)):
                sl = st % STAGES
                yield self.wait(0, "PV (CTA 0)", "full_v", sl=sl, st=st)
                for c in range(2):
                    assert self.v[c][sl][0] == (t, v, True), "products with other rows, or rows that were not patched"
                    self.v[c][sl][1] += 1
                self.commit("PV", "empty_v", sl, [self.v[0][sl], self.v[1][sl]])
                st += 1
            self.bars[0]["pv_sent"][eval(self.src.sent, {}, dict(t=t))].arrive()

            def made(t=t):
                self.o_tile = t
            self.later("PV", made)
            self.commit("PV", "pv_done", 0)
            t += 1

    def role_soft(self, cta, part, group):
        g = k = 0
        leader = self.bars[0]
        warps = 8 // self.GROUPS
        while True:
            item = yield from self.next_item(cta, k, warps, group)
            k += 1
            if item is None:
                return
            nt = self.tiles(item)
            for i in range(nt):
                t = g + i
                yield self.wait(cta, "softmax", "s_full", t=t)
                assert self.s[t & 1][0] == t, "logits of another tile"
                yield group.join()
                if self.vote[(cta, t)]:
                    yield group.join()
                assert self.s[t & 1][0] == t, "logits overwritten while they were read"
                self.s[t & 1][1] += 1
                leader["s_free"][t & 1].arrive(warps)
                if i > 0:
                    yield self.wait(cta, "softmax", "pv_done", 0, t=t)
                if t > 0:
                    assert self.o_tile == t - 1, "weights or output touched while products read them"
                self.p[cta][part] = t
                leader["p_full"][0].arrive(warps)
            yield group.join()
            g += nt
            if nt:
                yield self.wait(cta, "softmax", "pv_done", 1, g=g)
                assert self.o_tile == g - 1, "an output of another item"
                self.o_read += 1
                leader["o_free"][0].arrive(warps)
            yield group.join()
            self.done[cta * self.GROUPS + part].append(k - 1)

    # ---- a run
    def run(self):
        rng = self.rng
        self.vote = {(c, t): rng.random() < 0.5 for c in range(2) for t in range(sum(map(self.tiles, self.items)))}
        roles = {}
        for c in range(2):
            for name in ("items", "k", "v", "patch", "s", "pv"):
                roles[(name, c)] = getattr(self, "role_" + name)(c)
            soft = Group(self.GROUPS)
            for part in range(self.GROUPS):
                roles[("soft", c, part)] = self.role_soft(c, part, soft)
        blocked = {r: (lambda: True) for r in roles}
        speed = {r: 10 ** rng.uniform(-2.5, 0) for r in roles}       # some roles are far slower than others
        slow_copies, slow_s, slow_pv = (10 ** rng.uniform(-2.5, 0.5) for _ in range(3))
        while roles or self.queues:
            able = [(r, speed[r]) for r in roles if blocked[r]()]
            able += [(q, slow_s if q == "S" else slow_pv if q == "PV" else slow_copies) for q in self.queues]
            if not able:
                return "stuck: " + ", ".join(map(str, roles))
            pick = rng.choices([a for a, _ in able], [w for _, w in able])[0]
            if pick in self.queues:
                work = self.queues[pick]
                work.pop(0)()
                if not work:
                    del self.queues[pick]
                continue
            try:
                blocked[pick] = next(roles[pick])
            except StopIteration:
                del roles[pick]
        assert all(d == list(range(len(self.items))) for d in self.done)
        return "done"


def _items(rng, shape):
    """Blocks of a cluster's items: the last ones of a row set are often not clean."""
    def item(n):
        return [rng.random() < 0.6 for _ in range(n)]
    if shape == "short":                     # one tile of one block, the longest way between two items
        return [item(1) for _ in range(rng.randint(3, 8))]
    if shape == "long":
        return [item(rng.randint(5, 13)) for _ in range(rng.randint(2, 3))]
    return [item(rng.choice([0, 1, 1, 2, 4, 5, 8, 9])) for _ in range(rng.randint(3, 7))]


def outcomes(text, shape, runs):
    src = Source(text)
    got = []
    for seed in range(runs):
        rng = random.Random(f"{shape} {seed}")
        got.append(Cluster(src, _items(rng, shape), rng).run())
    return got


@pytest.mark.parametrize("shape", ["short", "long", "mixed"])
def test_no_order_of_the_roles_gets_stuck(shape):
    with open(SOURCE) as f:
        got = outcomes(f.read(), shape, 80)
    stuck = [g for g in got if g != "done"]
    assert not stuck, f"{len(stuck)} of {len(got)} orders, {stuck[0]}"


def test_the_model_sees_a_wait_that_misses_a_phase():
    """With one barrier for the PV products of even and odd tiles, the S issuer can come to its wait two
    phases late: the model has to get stuck."""
    with open(SOURCE) as f:
        text = f.read()
    one = re.sub(r"wait_warp\(&?pv_sent(\[[^\]]*\])?, .*?, abort_flag\)", "(t < 2 || wait_warp(pv_sent, t & 1, abort_flag))", text)
    one = re.sub(r"mbar_arrive\(&?pv_sent(\[[^\]]*\])?\)", "mbar_arrive(pv_sent)", one)
    got = outcomes(one, "short", 40)
    assert any(g.startswith("stuck") for g in got)
    assert "done" in got                     # what the timing of a run decides
