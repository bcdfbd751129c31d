"""The attention kernel's cut of a call's work, run on the CPU from the kernel's own header: a partition of every job, whose
pieces the joining kernel finds from what the parts write down about them."""
import os
import random
import subprocess

import pytest

from nvfp4_block_scaled_11_b200 import build as nvbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("cut") / "attention_cut")
    subprocess.run([nvbuild.NVCC, *nvbuild.ARCH, "-O1", "-std=c++17", "-o", exe, os.path.join(HERE, "c_abi", "attention_cut.cu")], check=True,
                   capture_output=True, text=True)

    def run(cases):
        """[(parts at most, jobs per sequence, costs)] -> [(total, n, J, M, starts, part of each unit, pieces)]."""
        text = "\n".join(f"{m} {j} {len(c)} " + " ".join(map(str, c)) for m, j, c in cases)
        lines = iter(subprocess.run([exe], input=text, check=True, capture_output=True, text=True, timeout=120).stdout.splitlines())
        out = []
        for _ in cases:
            head, starts, of = ([int(x) for x in next(lines).split()] for _ in range(3))
            pieces = []
            while (line := next(lines)) != "end":
                pieces.append(tuple(map(int, line.split())))
            out.append((*head, starts, of, pieces))
        return out
    return run


def test_the_cut_covers_every_job_once(cut):
    rnd = random.Random(0)
    J = cut([(1, 1, [100])])[0][2]
    cases = [(rnd.randrange(1, rnd.choice([8, 80, 400])), rnd.randrange(1, 5),
              [J + rnd.randrange(1, rnd.choice([2, 6, 40])) for _ in range(rnd.randrange(1, 12))]) for _ in range(400)]
    cases += [(444, 8, [J + 257] * 16), (148 * 3, 1, [J + 1] * 148 * 3), (65535, 1, [J + 1]), (7, 3, [J + 1] * 7)]
    for (most, jobs, costs), (total, n, j, m, starts, of, pieces) in zip(cases, cut(cases)):
        assert j == J and total == jobs * sum(costs) and 1 <= n <= most
        assert starts[0] == 0 and starts[-1] == total and n == max(1, min(most, total // m))
        sizes = [b - a for a, b in zip(starts, starts[1:])]
        assert max(sizes) - min(sizes) <= 1 and (n == 1 or min(sizes) >= m > J)     # a part is longer than a job's start
        assert all(starts[p] <= u < starts[p + 1] for u, p in enumerate(of))
        got = {}
        for part, b, job, first, last, begun, done in pieces:
            assert first < last
            got.setdefault((b, job), []).append((part, first, last, begun, done))
        begins, at = {}, 0
        for b, c in enumerate(costs):
            for job in range(jobs):
                ps = got.pop((b, job))
                # every unit of the job's work once, in order, by parts one after the other
                assert ps[0][1] == 0 and ps[-1][2] == c - J and all(x[2] == y[1] and y[0] == x[0] + 1 for x, y in zip(ps, ps[1:]))
                assert [x[3] for x in ps] == [1] + [0] * (len(ps) - 1) and [x[4] for x in ps] == [0] * (len(ps) - 1) + [1]
                if len(ps) > 1:
                    # the part that begins a cut job begins no other one, and tells the part that ends it
                    assert ps[0][0] not in begins and of[at + c - 1] == ps[-1][0]
                    begins[ps[0][0]] = (b, job)
                at += c
        assert not got
