"""What a kernel waits for before it leaves early (csrc/vp_waits.h), against a model of the barriers.

The header is plain C++: it is compiled for the host here, and its answers are
played through on a model of an mbarrier, for every state that a pair of CTAs
can be in when one of them gives up. Nothing of this runs on a GPU.
"""
import ctypes
import os
import re
import subprocess

import pytest

import vocab_wide_logprobs_gb300 as vp

CSRC = os.path.join(os.path.dirname(vp.__file__), "csrc")
NOTHING, ALL, NO_PEER, NO_LEADER = range(4)


@pytest.fixture(scope="module")
def header(tmp_path_factory):
    at = tmp_path_factory.mktemp("waits")
    source = at / "waits.cpp"
    source.write_text('#include "vp_waits.h"\n'
                      'extern "C" uint32_t late(uint32_t s, uint32_t a, uint32_t b, uint32_t n) {\n'
                      '    const vp::LateStage l = vp::late_stage(s, a, b, n);\n'
                      '    return l.owed << 1 | l.parity;\n}\n'
                      'extern "C" uint32_t next(uint32_t p, uint32_t b) { return vp::next_phase(p, b); }\n'
                      'extern "C" uint32_t word(uint32_t s, uint32_t l, uint32_t r) { return vp::fault_word(s, l, r); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(source), "-o",
                    str(at / "waits.so")], check=True)
    return ctypes.CDLL(str(at / "waits.so"))


class Barrier:
    """An mbarrier of one arrival: a phase ends when the arrival and all its bytes have come."""

    def __init__(self):
        self.phase, self.pending, self.tx = 0, 1, 0

    def arm(self, tx):
        assert self.pending == 1, "armed twice in a phase"
        self.pending, self.tx = 0, self.tx + tx
        self.turn()

    def land(self, tx):
        self.tx -= tx
        self.turn()

    def turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, 1

    def done(self, parity):
        return self.phase & 1 != parity


@pytest.mark.parametrize("n", [1, 3, 6, 10])
def test_every_copy_in_flight_is_awaited(header, n):
    """Both CTAs at every pair of counts, each copy under way or landed: the wait ends when the last has landed."""
    for used in range(3 * n + 1):                                    # fills whose both halves were used
        for leader in range(used, used + n + 1):                     # a stage is filled again only after that
            for peer in range(used, used + n + 1):
                for late in range(2):                                # of what is not used: all landed, all under way
                    bars, flying = [Barrier() for _ in range(n)], []
                    for f in range(max(leader, peer)):
                        for mine, tx in ((leader, "leader"), (peer, "peer")):
                            if f >= mine:
                                continue
                            if tx == "leader":
                                bars[f % n].arm(2)
                            if f >= used and late:
                                flying.append(f % n)
                            else:
                                bars[f % n].land(1)
                    plans = [divmod(header.late(s, leader, peer, n), 2) for s in range(n)]
                    for s, (owed, _) in enumerate(plans):
                        assert (owed == NOTHING) == (s >= max(leader, peer))
                        assert owed != NOTHING or s not in flying
                        if owed == NO_PEER:
                            bars[s].land(1)
                        if owed == NO_LEADER:
                            bars[s].arm(1)
                    for s, (owed, parity) in enumerate(plans):
                        assert owed == NOTHING or bars[s].done(parity) == (s not in flying)
                    for s in flying:
                        bars[s].land(1)
                    assert all(owed == NOTHING or bars[s].done(parity) for s, (owed, parity) in enumerate(plans))


def test_the_stage_that_is_waited_for_is_among_them(header):
    """The one whose copy is late holds up everything behind it: the producer stops right before filling it again."""
    assert header.late(2, 8, 8, 6) >> 1 == ALL                       # fill 8 would be stage 2's second
    assert header.late(2, 8, 9, 6) >> 1 == NO_LEADER and header.late(2, 9, 8, 6) >> 1 == NO_PEER


@pytest.mark.parametrize("name", ["vp_mxfp4.cu", "vp_gemm.cuh"])
def test_the_kernels_with_rings_ask(name):
    """The products of one CTA and of pairs, on every way out; and an accumulator is announced only when it is whole."""
    with open(os.path.join(CSRC, name)) as f:
        single, pair = re.split(r"\n\w*_pair_kernel\(const", f.read())
    assert "late_stage(" in single and "umma_commit(&bars.done);" in single
    assert "pair_ring_used<" in pair and "pair_ends<" in pair and "umma_commit_pair_here(&bars.done);" in pair
    for kernel in (single, pair):
        lines = [line.split("//")[0].strip() for line in kernel.splitlines()]
        at = [i for i, line in enumerate(lines) if re.match(r"umma_commit(_pair)?\(&bars\.acc_full", line)]
        assert len(at) == 1 and lines[at[0] - 1] == "if (!ok) break;"


def tiles_of_a_cta(header, copied, late, sees, stops=True):
    """The rules' loop over tiles: the thread that begins the copies and another one.

    copied[i]: tile i comes by a bulk copy. The late-th lands while it is waited for; sees: which of the two threads'
    waits ended all the same. Returns how many waits ran out in all."""
    bars = [Barrier(), Barrier()]
    arrived, parity, ran_out, flying = [True, True], [0, 0], 0, set()

    def stage(i):
        if copied[i] and (arrived[0] or not stops):
            bars[i % 2].arm(1)
            flying.add(i)

    def lands(but=None):
        for i in flying - {but}:
            bars[i % 2].land(1)
            flying.discard(i)

    stage(0)
    for i in range(len(copied)):
        buf = i % 2
        if i + 1 < len(copied):
            stage(i + 1)
        if i == late:
            first = [t for t in range(2) if not sees[t]]
        else:
            lands(but=late if late is not None and i < late else None)
            first = []
        for t in first + [t for t in range(2) if t not in first]:
            if i == late and t not in first:
                lands()
            if not copied[i] or not (arrived[t] or not stops):
                continue
            if not bars[buf].done(header.next(parity[t], buf)):
                ran_out += 1
                arrived[t] = False
                assert stops or t
                waits = [(buf, header.next(parity[t], buf))]
                if i + 1 < len(copied) and copied[i + 1]:
                    waits.append((buf ^ 1, header.next(parity[t], buf ^ 1)))
                if t == 0:                                           # the thread that began them sees all land
                    assert {b for b, _ in waits} == {k % 2 for k in flying}
                    lands()
                    assert all(bars[b].done(p) for b, p in waits)
            parity[t] ^= 1 << buf
    assert not flying                                                # nothing is under way at the end
    return ran_out


def test_a_late_tile_of_the_rules(header):
    """No barrier is armed in an open phase, all copies land before the CTA ends, and few waits run out on the way."""
    for k in range(128):
        copied = [bool(k >> i & 1) for i in range(7)]
        assert tiles_of_a_cta(header, copied, late=None, sees=(True, True)) == 0
        for late in (i for i in range(7) if copied[i]):
            for sees in ((True, True), (True, False), (False, True), (False, False)):
                ran_out = tiles_of_a_cta(header, copied, late, sees)
                assert ran_out <= 2 and (ran_out > 0 or all(sees))
    with pytest.raises(AssertionError):                              # going on as if nothing had happened
        tiles_of_a_cta(header, [True] * 7, 2, (False, False), stops=False)


def test_the_rules_stop_their_copies():
    with open(os.path.join(CSRC, "vp_rules.cu")) as f:
        source = f.read()
    assert len(re.findall(r"if \(tid == 0 && arrived[^)]*\)?\)? copy\(", source)) == 2
    assert "if (staged.bulk && arrived) {" in source and "next_phase(parity, buf ^ 1)" in source


def test_the_fault_word_says_whose_outputs_are_void(header):
    words = {(scans, products, rules): header.word(scans, products, rules)
             for scans in range(4) for products in range(8) for rules in range(2)}
    assert len(set(words.values())) == len(words) and words[0, 0, 0] == 0
    assert words[1, 0, 0] == 1 and words[0, 4, 0] == 16 and words[0, 0, 1] == 32
    with open(os.path.join(CSRC, "vp_api.cu")) as f:
        assert "vp::fault_word(" in f.read()
