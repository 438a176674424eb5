"""The measured cases of the drafter's operators: draws stay inside what the operators take, and the kernels agree with the
64-bit forms on small ones."""
import importlib.util
import math
import os
import random

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests.target_ref import U32, half_step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    return ops


def test_cases_and_draws_are_well_formed():
    ops = load()
    rng = random.Random(11)
    cases = ops.listed() + [ops.draw(rng) for _ in range(200)]
    names = [c["name"] for c in ops.listed()]
    assert 4 <= len(names) <= 12 and len(set(names)) == len(names)
    assert {c["op"] for c in cases[len(names):]} == {"sample", "append8", "attn8", "sinks"}
    for c in cases:
        w = ops.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
        if c["op"] == "sample":
            assert 1 <= c["V"] <= 262144 and c["N"] >= 1 and 0 <= c["top_k"] and c["dtype"] in ("bf16", "f32")
            continue
        assert c["page"] % 16 == 0 and c["Hq"] % c["Hkv"] == 0 and c["D"] in (64, 128) and c["dtype"] in ("bf16", "f16")
        past, new = ops._spread(c)
        assert max(new) == c["N"] and min(new) >= 1 and min(past) >= 0 and len(past) == len(new) == c["B"]
        if c["op"] == "append8":
            assert c["rot"] % 16 == 0 and c["rot"] <= c["D"]
        else:
            assert c["window"] >= (c["op"] == "sinks") and c["sinks"] >= 0
            assert sv.attention_workspace_size(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]) > 0
            # visible pairs and keys, counted one by one
            n, p = min(new[0], 50), past[0]
            if p < 3000:
                seen = [[j for j in range(p + i + 1) if not c["window"] or j > p + i - c["window"] or j < c["sinks"]]
                        for i in range(n)]
                assert ops._visible(p, n, c["window"], c["sinks"])[0] == sum(map(len, seen))


def small(ops, op, count):
    rng = random.Random(sum(map(ord, op)))
    res = []
    while len(res) < count:
        c = ops.draw(rng)
        if c["op"] != op:
            continue
        if op == "sample":
            if c["B"] * c["N"] <= 48 and c["B"] * c["N"] * c["V"] < 2e6:
                res.append(c)
            continue
        past, new = ops._spread(c)
        if (sum(past) + sum(new)) * c["Hkv"] * c["D"] < 3e7 and ops.work(c)["flops"] < 2e9 and c["B"] <= 16:
            res.append(c)
    return res


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["sample", "append8", "attn8", "sinks"])
def test_kernels_agree_with_the_definitions_on_draws(op):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops = load()
    ops.own = True
    for n, c in enumerate(small(ops, op, 12)):
        s = ops.prepare(c, 100 + n)
        got, want = ops.run(s), ops.exact(c, 100 + n)
        if op == "sample":
            assert torch.equal(got[0], want[0]), c
            assert bool(((got[1].double() - want[1]).abs() <= want[1] * U32 * 1.01).all()), c
            continue
        if op == "append8":
            assert torch.equal(got[1].double(), want[1]) and torch.equal(got[2].double(), want[2]), c
            h = half_step(got[0].dtype)
            # two products and their sum in 32 bits of two elements of a head, then one rounding
            tol = want[0].abs() * h + (1 + h) * 3 * U32 * 2 * s["q"].double().abs().amax(-1, keepdim=True)
            if c["dtype"] == "f16":
                tol = tol + 2.0 ** -25
            assert bool(((got[0].double() - want[0]).abs() <= tol).all()), c
            continue
        # As tests/drafter_ref.py's bound, with the largest of all values and scores in place of a row's own
        dt = s["q"].dtype
        eight = op == "attn8"
        D, L = c["D"], s["max_context"]
        k, v = s["k_pages"].double(), s["v_pages"].double()
        if eight:
            k, v = (x.reshape(*x.shape[:2], -1, 16, D) * s[n_].double()[..., None, None]
                    for x, n_ in ((k, "k_scales"), (v, "v_scales")))
        big = float(v.abs().max())
        top = float(s["q"].double().norm(dim=-1).max()) * float(k.norm(dim=-1).max()) / math.sqrt(D)
        h = half_step(torch.float16 if eight else dt)
        delta = top * (2 * D + 8) * U32
        tol = big * (h * (1 + eight * 2.0 ** -8) + 2 * delta + 4 * (L + 64) * U32) + half_step(dt) * want.abs() + 1e-30
        if dt == torch.float16:
            tol = tol + 2.0 ** -25
        if eight or dt == torch.float16:
            tol = tol + 2.0 ** -30 * L * big
        assert bool(((got.double() - want).abs() <= tol).all()), c
