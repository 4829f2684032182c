"""exl3_rotary into outputs that lie beside its inputs or over them."""
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_outputs_beside_and_over_the_inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens, heads, kv, dim = 41, 6, 2, 64
    wide = torch.randn((tokens, 2 * (heads + kv), dim), generator=g, device="cuda").half()
    position = torch.randint(0, 9000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    f = B.exl3_rotary_freqs(dim)
    q, k = wide[:, :heads], wide[:, heads:heads + kv]
    want = B.exl3_rotary(q, k, position, f)
    other = wide[:, heads + kv:]                       # the rest of the same rows
    B.exl3_rotary(q, k, position, f, q_out=other[:, :heads], k_out=other[:, heads:])
    assert torch.equal(other[:, :heads], want[0]) and torch.equal(other[:, heads:], want[1])
    one = wide[:1].clone()
    B.exl3_rotary(one[:, :heads], one[:, heads:heads + kv], position[:1], f, q_out=one[:, :heads], k_out=one[:, heads:heads + kv])
    assert torch.equal(one[:, :heads], want[0][:1]) and torch.equal(one[:, heads:heads + kv], want[1][:1])
    before = wide.clone()
    dense = wide.view(-1)[:tokens * heads * dim].view(tokens, heads, dim)            # q's first bytes, of another stride
    for q_out, k_out in ((dense, None), (q, q[:, :kv]), (other[:, :heads], other[:, 1:1 + kv]), (wide[:, 1:1 + heads], None), (wide[:, kv:kv + heads], k)):
        with pytest.raises(B.Exl3Error):
            B.exl3_rotary(q, k, position, f, q_out=q_out, k_out=k_out)
    assert torch.equal(wide, before)
    B.exl3_rotary(q, k, position, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_as_many_tokens_as_have_a_number():
    tokens, dim = 2 ** 31 - 1, 16
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free memory")
    q = torch.empty((tokens, 1, dim), dtype=torch.float16, device="cuda")
    position = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    some = torch.cat([torch.arange(300), 2 ** 30 + torch.arange(300), tokens - 300 + torch.arange(300)]).cuda()
    small = torch.randn((900, 1, dim), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    where = torch.arange(900, dtype=torch.int32, device="cuda") * 7
    q[some], position[some] = small, where
    f = B.exl3_rotary_freqs(dim)
    B.exl3_rotary(q, None, position, f, q_out=q)
    assert torch.equal(q[some], B.exl3_rotary(small, None, where, f)[0])
    del q, position
    torch.cuda.empty_cache()
