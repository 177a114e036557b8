"""The Python binding of the attention calls: whose memory a call uses, and what it checks before it launches."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import Paged, S, check_attention, prompt_inputs, ref_prompt  # noqa: F401  (S: the library)


def stream_of(t):
    """The stream that the caching allocator keeps t's memory for."""
    a = t.untyped_storage().data_ptr()
    return next(g["stream"] for g in torch.cuda.memory_snapshot() if g["address"] <= a < g["address"] + g["total_size"])


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [False, True])
def test_what_a_call_makes_belongs_to_its_launch_stream(S, monkeypatch, as_int):  # noqa: F811
    """With stream= and nothing brought along, outputs and workspace are memory of that stream: on the
    current one the workspace's zero fill would not be ordered before the kernels, and its memory would be handed out
    again while they run."""
    p = Paged(S, [200, 31], [4, 9], 8, 2, 128, 16, "bf16", 12)
    lens = [90, 200]
    qkv, cu = prompt_inputs(lens, 8, 2, 128, 13)
    dev, cud = qkv.cuda(), cu.cuda()
    made = []
    alloc = S.alloc_attn_workspace

    def keep(*a, **kw):
        made.append(alloc(*a, **kw))
        return made[-1]

    monkeypatch.setattr(S, "alloc_attn_workspace", keep)
    table = S.rope_table(256, 128)
    pos = torch.arange(290, device="cuda").int() % 256
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    st = side.cuda_stream if as_int else side
    tree = p.call(S, stream=st)
    torch.cuda.synchronize()  # its inputs were temporaries of the current stream
    prompt = S.attn_prompt(dev[:, :8], dev[:, 8:10], dev[:, 10:], cud, stream=st)
    q, k = S.qk_norm_rope(dev[:, :8], dev[:, 8:10], None, table, pos, stream=st)
    torch.cuda.synchronize()
    assert len(made) == 3
    for t in (*made, tree, prompt, q, k):
        assert stream_of(t) == side.cuda_stream
    p.check(tree)
    check_attention(prompt.cpu(), *ref_prompt(qkv, lens, 8, 2, 128), 128, 200, True)
    # without stream=, the current stream's
    with torch.cuda.stream(side):
        here = S.attn_prompt(dev[:, :8], dev[:, 8:10], dev[:, 10:], cud)
    assert stream_of(here) == side.cuda_stream
    assert stream_of(S.attn_prompt(dev[:, :8], dev[:, 8:10], dev[:, 10:], cud)) == torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()


def test_a_workspace_in_host_memory_is_refused(S):  # noqa: F811
    with pytest.raises(S.SffnError) as e:
        S._space(torch.zeros(256, dtype=torch.uint8), "here")
    assert e.value.status == S.ERR_WORKSPACE


@pytest.mark.gpu
def test_workspaces_that_a_call_takes(S):  # noqa: F811
    """Refused before anything is launched: host memory, every other element of an array.  Taken: an
    array of another type whose bytes are enough, which is measured in bytes."""
    p = Paged(S, [20], [2], 4, 2, 64, 16, "bf16", 1)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    k, cu = q[:, :2].contiguous(), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    need = S.attn_workspace_size(S.WS_ATTN_TREE, 2, 1, 4, 2, 64)
    pos = torch.arange(3, device="cuda").int()
    for ws in (torch.zeros(need, dtype=torch.uint8), torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        for call in (lambda: p.call(S, workspace=ws), lambda: S.attn_prompt(q, k, k, cu, workspace=ws),
                     lambda: S.qk_norm_rope(q, k, None, S.rope_table(4, 64), pos, workspace=ws)):
            with pytest.raises(S.SffnError) as e:
                call()
            assert e.value.status == S.ERR_WORKSPACE
    p.check(p.call(S, workspace=torch.zeros(need // 4, dtype=torch.int32, device="cuda")))
    with pytest.raises(S.SffnError):
        p.call(S, workspace=torch.zeros(need // 4 - 64, dtype=torch.int32, device="cuda"))
