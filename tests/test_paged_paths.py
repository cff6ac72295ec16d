"""Every way in which the host cuts an attention call over the paged cache has
a case that the GPU tests hold against the oracle: the choice made for each
case of paged_paths.PATHS is the one that the case is there for (compiles
tests/native/shared_rule_check.cpp; no GPU needed)."""
import pathlib
import shutil
import subprocess

import pytest

from paged_paths import AHEAD, FEW, NONE, PASS, PATHS

ROOT = pathlib.Path(__file__).resolve().parents[1]
SMS = 148


def choices(exe, calls):
    """The host's choice for calls (nq, nkv, hd, page, P, lens, new, window), padding rows."""
    lines = []
    for (nq, nkv, hd, page, P, lens, new, window), pad in calls:
        width = max(1, max(-(-n // page) for n in lens)) + 1  # as the cases' tables have it
        lines.append([sum(new) + pad, len(lens), nq, nkv, hd, page, width, P, window, max(1, max(new)), SMS])
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, x)) for x in lines), capture_output=True, text=True,
                       timeout=60)
    out = []
    for (call, _), line in zip(calls, r.stdout.split("\n")):
        few, many, ahead, pf, ns, rest, own, final = map(int, line.split())
        out.append(dict(few=few, many=bool(many), prefix=FEW if pf else AHEAD if ahead else PASS if call[4] else NONE,
                        pieces=ns, gap=rest < ns, own=own, final=bool(final)))
    return out


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path_factory.mktemp("rule") / "shared_rule_check"
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", str(ROOT / "w4_weight_only_b200" / "csrc"),
                        str(ROOT / "tests" / "native" / "shared_rule_check.cpp"), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


def test_cases_are_on_their_paths(rule):
    got = choices(rule, [(call, pad) for call, pad, _ in PATHS.values()])
    for (name, (_, _, want)), have in zip(PATHS.items(), got):
        assert {k: have[k] for k in want} == want, name


def test_every_path_has_a_case(rule):
    got = choices(rule, [(call, pad) for call, pad, _ in PATHS.values()])
    window = [call[7] > 0 for call, _, _ in PATHS.values()]
    for w in (False, True):
        have = [g for g, x in zip(got, window) if x == w]
        for prefix in (FEW, PASS, AHEAD):
            assert any(g["prefix"] == prefix for g in have), (prefix, w)
        assert any(g["prefix"] == PASS and g["gap"] for g in have), w
        assert any(g["prefix"] == PASS and g["many"] and g["final"] and g["pieces"] > 1 for g in have), w
        assert any(g["prefix"] == AHEAD and g["final"] for g in have), w
    assert any(g["prefix"] == PASS and g["many"] and not g["final"] and g["own"] > 1 for g in got)
    assert {g["few"] for g in got if g["prefix"] == FEW} == {16, 32, 48}
