"""Refusals of the operators' wrappers and steps, and what their plans look
like, on the CPU (no kernel runs)."""
import os
import subprocess
import sys

import pytest
import torch

import operators_common as oc
from paged_kv_cache_16_gb300 import binding, build, workloads
from paged_kv_cache_16_gb300.step import DeviceStep, GraphStep


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("call", ["pa_attention_scaled", "pa_attention_scaled_launch"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("change,message", [
    (lambda a: dict(kc=a["kc"].view(torch.uint8 if a["kc"].dtype == torch.int8 else torch.int8),
                    vc=a["vc"].view(torch.uint8 if a["vc"].dtype == torch.int8 else torch.int8)), "type of codes"),
    (lambda a: dict(out=a["out"][:-1]), "rows"), (lambda a: dict(q=a["q"][:-1]), "rows"),
    (lambda a: dict(table=a["table"][:-1]), "requests"), (lambda a: dict(table=a["table"][:, :-1].contiguous()), "blocks each"),
    (lambda a: dict(kc=a["kc"][:-1], vc=a["vc"][:-1], ks=a["ks"][:-1], vs=a["vs"][:-1]), "caches"),
    (lambda a: dict(kc=a["kc"].view(-1, 16, 4, 64), vc=a["vc"].view(-1, 16, 4, 64), ks=a["ks"].repeat(1, 2),
                    vs=a["vs"].repeat(1, 2)), "caches"),
    (lambda a: dict(kc=a["kc"].view(-1, 8, 2, 128), vc=a["vc"].view(-1, 8, 2, 128), ks=a["ks"].repeat(2, 1),
                    vs=a["vs"].repeat(2, 1)), "caches")])
def test_attention_refuses_what_its_plan_was_not_made_for(call, code, change, message):
    """The kernels read and write by the plan's sizes: an output of fewer rows would
    be written past its end, int8 codes read as E4M3 ones."""
    c = oc.Case(hq=4, hkv=2, d=128, q_lens=[3, 1], seq_lens=[40, 90], code=code)
    plan = binding.pa_plan(**c.desc(num_sms=4))
    a = dict(q=c.q, kc=c.kc, vc=c.vc, ks=c.ks, vs=c.vs, table=torch.from_numpy(c.table), out=torch.empty_like(c.q),
             workspace=torch.zeros(plan.workspace_bytes, dtype=torch.uint8))
    with pytest.raises(ValueError, match=message):
        getattr(binding, call)(plan, *(a | change(a)).values())
    with pytest.raises(ValueError, match="current CUDA device"):     # the last check, reached by the plan's own tensors
        getattr(binding, call)(plan, *a.values())
    more = dict(a, q=torch.cat([c.q, c.q]), out=torch.empty(9, 4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="current CUDA device"):     # rows behind the last are the caller's
        getattr(binding, call)(plan, *more.values())


def test_attention_of_a_fixed_shape_wants_its_capacity():
    c = oc.Case(hq=4, hkv=2, d=64, q_lens=[1, 1], seq_lens=[40, 90], code="int8")
    plan = binding.pa_plan_fixed(max_tokens=8, max_reqs=4, **c.desc(num_sms=4))
    a = dict(q=c.q, kc=c.kc, vc=c.vc, ks=c.ks, vs=c.vs, table=torch.from_numpy(c.table), out=torch.empty_like(c.q),
             workspace=torch.zeros(plan.workspace_bytes, dtype=torch.uint8))
    with pytest.raises(ValueError, match="rows"):
        binding.pa_attention_scaled_launch(plan, *a.values())
    a["q"] = a["out"] = torch.empty(8, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        binding.pa_attention_scaled_launch(plan, *a.values())


def append_call(**over):
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[3, 1], computed=[5, 0], code="int8")
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32)  # noqa: E731
    a = dict(rope=None, key=c.key, value=c.value, query_start_loc=i32(c.qsl), num_computed=i32(c.nc),
             block_table=i32(c.table), key_cache=c.kc, value_cache=c.vc, key_scales=c.ks, value_scales=c.vs)
    return binding.pa_append_kv(**(a | over))


@pytest.mark.parametrize("word", [torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64),
                                  torch.zeros(0, dtype=torch.int32)])
def test_append_refuses_error_words_of_other_types(word):
    """The kernel sets bits of four bytes there."""
    with pytest.raises(ValueError, match="device_error_word"):
        append_call(device_error_word=word)
    with pytest.raises(ValueError, match="rows, starts"):
        append_call(device_error_word=torch.zeros(1, dtype=torch.int32))


def test_append_refuses_a_destroyed_rope():
    """It must not pass for no rope at all, with which keys are stored unrotated."""
    rope = binding.pa_rope_create(rotary_dim=64)
    with pytest.raises(ValueError, match="rows, starts"):
        append_call(rope=rope)
    rope.destroy()
    with pytest.raises(ValueError, match="destroyed"):
        append_call(rope=rope)


def small_batch(kind):
    return workloads.make_batch(name="cpu", num_heads_q=4, num_heads_kv=2, head_dim=128, q_lens=[1, 3], seq_lens=[20, 33],
                                num_blocks=8, kv_cache_dtype=kind)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("call", ["run", "run_fused", "write"])
def test_step_with_a_rope_refuses_calls_that_do_not_rotate(kind, call):
    b = small_batch(kind)
    st = DeviceStep(b, "cpu", num_sms=4, rope=binding.pa_rope_create(rotary_dim=64))
    args = (b.q, b.key, b.value, b.key_cache, b.value_cache)
    with pytest.raises(ValueError, match="run_append"):
        getattr(st, call)(*args[call == "write":])


@pytest.mark.parametrize("kind", ["int8_block", "fp8_block", "fp8", "bf16"])
def test_steps_refuse_scales_that_do_not_go_with_their_caches(kind):
    """Codes of a block-scaled cache without its scales would be written as E4M3
    codes with one scale, and the reverse."""
    b = small_batch(kind)
    scales = (torch.ones(8, 2), torch.ones(8, 2))
    bad = [(None, None), (scales[0], None), (None, scales[1])] if "block" in kind else [scales, (scales[0], None)]
    st = DeviceStep(b, "cpu", num_sms=4)
    gs = GraphStep(num_heads_q=4, num_heads_kv=2, head_dim=128, num_blocks=8, max_blocks_per_req=3,
                   softmax_scale=b.softmax_scale, max_tokens=8, max_reqs=4, kv_cache_dtype=kind, num_sms=4, device="cpu")
    rows = (b.q, b.key, b.value, b.key_cache, b.value_cache)
    for s in bad:
        for call in (lambda: st.append(*rows, *s), lambda: st.run_append(*rows, *s), lambda: gs.run(b, *rows, *s),
                     lambda: gs.capture(None, *rows[3:], *s), lambda: gs.enqueue(None, *rows[3:], None, *s)):
            with pytest.raises(ValueError, match="scales"):
                call()


def test_binding_without_torch():
    """Plans, their metadata and rotations do not need torch."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from paged_kv_cache_16_gb300 import binding\n"
            "p = binding.pa_plan(num_heads_q=4, num_heads_kv=2, head_dim=64, num_blocks=9, query_start_loc=[0, 1],\n"
            "                    seq_lens=[20], num_computed_tokens=[19], max_blocks_per_req=2, softmax_scale=0.1, num_sms=4)\n"
            "assert p.info()['num_tokens'] == 1 and binding.pa_plan_metadata_bytes(p) > 0\n"
            "assert binding.pa_rope_create(rotary_dim=8).frequencies()[1] == 1.0\n")
    subprocess.run([sys.executable, "-c", code], check=True,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("name", ["auto", "bfloat16"])
def test_other_cache_type_names_are_bf16(name):
    a, b = small_batch("bf16"), small_batch(name)
    for x, y in ((a.key_cache, b.key_cache), (a.value_cache, b.value_cache)):
        assert y.dtype == torch.bfloat16 and torch.equal(x, y)
    assert b.key_scales is None and DeviceStep(b, "cpu", num_sms=4).plan.workspace_bytes == \
        DeviceStep(a, "cpu", num_sms=4).plan.workspace_bytes
    gs = GraphStep(num_heads_q=4, num_heads_kv=2, head_dim=128, num_blocks=8, max_blocks_per_req=3, softmax_scale=0.1,
                   max_tokens=8, max_reqs=4, kv_cache_dtype=name, num_sms=4, device="cpu")
    assert gs.model["kv_cache_dtype"] == binding.PA_KV_BF16
