"""Segmented products that take a workspace, on a stream of their own: what they
allocate belongs to that stream, so work on other streams cannot reuse it."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _segments as ref

pytestmark = pytest.mark.gpu


def _group(gen):
    ids = torch.randint(-1, 40, (20000,), generator=gen, device="cuda")  # past one workgroup's rows
    assert g.lib().gemm_f16_group_rows_workspace(20000, 40) > 0
    return lambda **k: g.group_rows(ids, 40, **k)


def _tn(gen):
    off = ref.offsets_of([6000, 0, 3500]).cuda()
    a, b = ref.eighths(gen, 9500, 200), ref.eighths(gen, 9500, 136)
    assert g.lib().gemm_f16_grouped_tn_workspace(9500, 3, 136, 200) > 0
    return lambda **k: (g.gemm_f16_grouped_tn(a, b, off, **k),)


def _lora(rows):
    def make(gen):
        ids = torch.randint(-1, 3, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        order, _, off = g.group_rows(ids, 3)
        t = [ref.normal(gen, *s) for s in ((rows, 512), (384, 512), (3, 16, 512), (3, 384, 16))]
        return lambda **k: (g.gemm_f16_lora_nt(*t, ids, order, off, **k),)
    return make


@pytest.mark.parametrize("make", [_group, _tn, _lora(5), _lora(50), _lora(300)],
                         ids=["group", "tn", "lora5", "lora50", "lora300"])
def test_a_workspace_belongs_to_the_calls_stream(make):
    call = make(torch.Generator(device="cuda").manual_seed(4))
    want = [t.clone() for t in call()]
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (side, third):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = []
        for s in (side, third, side):  # two streams in flight, the default one overwriting what it gets
            got.append(call(stream=s))
            junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(4)]
            del junk
        torch.cuda.synchronize()
        for out in got:
            for have, expect in zip(out, want):
                assert torch.equal(have, expect)


def test_a_threads_calls_do_not_meet():
    import threading

    calls = [make(torch.Generator(device="cuda").manual_seed(i)) for i, make in enumerate((_tn, _lora(50), _lora(300)))]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    off = []

    def work(c, expect):
        s = torch.cuda.Stream()
        for _ in range(5):
            got = c(stream=s)
            s.synchronize()
            off.extend(1 for a, b in zip(got, expect) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not off
