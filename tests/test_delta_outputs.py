"""Outputs of the gated delta rule and of the block norm that start where an input or another output does: one would be
written over the other, so the calls are refused (no GPU: nothing is launched)."""
from __future__ import annotations

import itertools

import pytest

import mamba2_ssd_selective_gb300 as ssd
from tests.test_delta_abi import INVALID, _built, big, bn_dims, dr_dims, refused  # noqa: F401

INPUTS = {n: (1 + i) << 16 for i, n in enumerate(("q", "k", "v", "log_decay", "beta", "initial_states", "cu_seqlens", "dout",
                                                  "dfinal_states", "slot_idx"))}
OUT = {n: (33 + i) << 16 for i, n in enumerate(("o", "final_states", "dq", "dk", "dv", "dlog_decay", "dbeta",
                                                "dinitial_states", "states"))}
PAIR = dict(nseq=2, packed=1, seqlen=0, total_tokens=200)


def rule(call, **at):
    """A call whose outputs are at addresses of their own, but for those given."""
    at = {**INPUTS, **OUT, **at}
    step = call == "step"
    dims = dr_dims(seqlen=1) if step else dr_dims(**PAIR)
    inputs = ssd.SsdDeltaRuleInputs(at["q"], 128, at["k"], 128, at["v"], 256, at["log_decay"], 4, at["beta"], 4,
                                    None if step else at["initial_states"], None if step else at["cu_seqlens"], 1.0, 1e-6)
    if step:
        return ssd.ssd_delta_rule_step, dims, inputs, at["states"], 2, at["slot_idx"], at["o"], 256
    if call == "forward":
        return ssd.ssd_delta_rule_forward, dims, inputs, at["o"], 256, at["final_states"], *big(dims, False)
    grads = ssd.SsdDeltaRuleGrads(at["dq"], 128, at["dk"], 128, at["dv"], 256, at["dlog_decay"], 4, at["dbeta"], 4,
                                  at["dinitial_states"])
    return ssd.ssd_delta_rule_backward, dims, inputs, at["dout"], 256, at["dfinal_states"], grads, *big(dims, True)


READ = ("q", "k", "v", "log_decay", "beta")
RULE = ([("forward", "o", n) for n in (*READ, "initial_states", "cu_seqlens", "final_states")] +
        [("forward", "final_states", n) for n in (*READ, "cu_seqlens")] +
        [("step", "o", n) for n in (*READ, "slot_idx", "states")] + [("step", "states", n) for n in (*READ, "slot_idx")] +
        [("backward", o, n) for o in ("dq", "dk", "dv", "dlog_decay", "dbeta", "dinitial_states")
         for n in (*READ, "initial_states", "cu_seqlens", "dout", "dfinal_states")] +
        [("backward", *p) for p in itertools.combinations(("dq", "dk", "dv", "dlog_decay", "dbeta", "dinitial_states"), 2)])


@pytest.mark.parametrize("call,out,other", RULE)
def test_delta_rule(call, out, other):
    refused(INVALID, *rule(call, **{out: {**INPUTS, **OUT}[other]}))


NORM_IN = {n: (1 + i) << 16 for i, n in enumerate(("x", "z", "residual", "post_weight", "branch_scale", "pre_weight", "h", "dh",
                                                   "dy", "rstd_post", "rstd_pre"))}
NORM_OUT = {n: (33 + i) << 16 for i, n in enumerate(("h", "y", "rstd_post", "rstd_pre", "dx", "dz", "dresidual", "dpost_weight",
                                                     "dbranch_scale", "dpre_weight"))}
WEIGHTS = ("post_weight", "branch_scale", "pre_weight")


def norm(call, **at):
    out = {n: at.get(n, p) for n, p in NORM_OUT.items()}
    d, i = bn_dims(), NORM_IN
    inputs = ssd.SsdBlockNormInputs(i["x"], 64, i["z"], 64, i["residual"] if call == "forward" else None, 64,
                                    *(i[w] for w in WEIGHTS), 1e-6)
    if call == "forward":
        return ssd.ssd_block_norm_forward, d, inputs, out["h"], 64, out["y"], 64, out["rstd_post"], out["rstd_pre"]
    saved = ssd.SsdBlockNormSaved(i["h"], 64, i["dh"], 64, i["dy"], 64, i["rstd_post"], i["rstd_pre"])
    grads = ssd.SsdBlockNormGrads(out["dx"], 64, out["dz"], 64, out["dresidual"], 64,
                                  *(out["d" + w] for w in WEIGHTS))
    return (ssd.ssd_block_norm_backward, d, inputs, saved, grads, 1 << 20, ssd.ssd_block_norm_workspace_size(d))


FORWARD, GRADS = ("h", "y", "rstd_post", "rstd_pre"), ("dx", "dz", "dresidual", *("d" + w for w in WEIGHTS))
NORM = ([("forward", o, n) for o in FORWARD for n in ("x", "z", "residual", *WEIGHTS) if (o, n) != ("h", "residual")] +
        [("forward", a, NORM_OUT[b]) for a, b in itertools.combinations(FORWARD, 2)] +
        [("backward", o, n) for o in GRADS[:3] for n in ("x", "z", *WEIGHTS, "h", "dh", "dy", "rstd_post", "rstd_pre")
         if (o, n) != ("dresidual", "dh")] +
        [("backward", a, NORM_OUT[b]) for a, b in itertools.combinations(GRADS, 2)])


@pytest.mark.parametrize("call,out,other", NORM)
def test_block_norm(call, out, other):
    refused(INVALID, *norm(call, **{out: NORM_IN[other] if isinstance(other, str) else other}))
