"""Calls of the gated recurrence and the norms as programs make them (needs an
MI355X): tensors in the wrong place beside a stream."""
import pytest
import torch

import selective_state_space_65_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_host_tensors_beside_a_stream():
    """A tensor left on the host is refused by name, with a stream as without one."""
    x, state = torch.randn((2, 6, 300), device=DEV), torch.randn((2, 6), device=DEV)
    tok = x[..., 0].contiguous()
    _, _, ck = ssm.gated_scan_fwd_save(x, x)
    _, _, mean, rstd = ssm.norm_fwd(tok)
    side = torch.cuda.Stream()
    for stream in (None, side):
        for name, call in (("gate", lambda: ssm.gated_scan_fwd(x, x.cpu(), stream=stream)),
                           ("z", lambda: ssm.gated_scan_fwd_save(x, x, z=x.cpu(), stream=stream)),
                           ("dy", lambda: ssm.gated_scan_bwd(x, x, x.cpu(), ck, stream=stream)),
                           ("gate", lambda: ssm.gated_state_update(state, tok, tok.cpu(), stream=stream)),
                           ("residual", lambda: ssm.norm_fwd(tok, residual=tok.cpu(), stream=stream)),
                           ("rstd", lambda: ssm.norm_bwd(tok, tok, rstd.cpu(), mean=mean, stream=stream))):
            with pytest.raises(ValueError, match=name + ": expected device"):
                call()
    torch.cuda.synchronize()
