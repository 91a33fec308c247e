"""Status codes of failed CUDA calls: BSC_ERR_CUDA for every one, in every entry point (BSC_ERR_UNSUPPORTED is for arguments
and devices, which are checked before a launch)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_causal_gb300", "csrc")


def test_failed_cuda_calls_are_cuda_errors():
    with open(os.path.join(CSRC, "api.cu")) as f:
        api = f.read()
    body = re.search(r"bsc_status from_cuda\(cudaError_t e\) \{(.*?)\n?\}\n", api, flags=re.S).group(1)
    assert re.findall(r"BSC_\w+", body) == ["BSC_OK", "BSC_ERR_CUDA"]
    for name in os.listdir(CSRC):       # and no launch passes an argument's refusal off as one
        with open(os.path.join(CSRC, name)) as f:
            assert "cudaErrorNotSupported" not in f.read(), name
